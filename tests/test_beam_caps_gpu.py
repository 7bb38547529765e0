"""A beam search's selection under softcaps of every size, against its definition in 64 bits.

Tolerance of a score. Up to cap * scale = 1024 an exponent is off by 2^-21 of cap * scale, as in test_beam_gpu, and
the sum by 2^-17. Above, the exponents are taken from z(x) - z(top), to 2^-19 of it: p_i being the terms' shares, the
sum is off by 2^-19 sum p_i |d_i| of itself at most, where sum p_i |d_i| <= log V (it is the shares' entropy less
-log p_top); and its additions by 2^-17 as ever."""
import math

import pytest
import torch

import gradient_row_online_gb300 as pkg

pytestmark = pytest.mark.gpu

ROWS, V = 6, 20000


def body(cap, size, dtype, g):
    """Logits some way (`size` caps) from zero, on either side or both."""
    x = 3.0 * torch.randn(ROWS, V, generator=g)
    at = min(size * cap, 1e38)
    x[:4] += at * torch.tensor([1.0, -1.0, 0.5, -0.5])[:, None]
    x[4] += at * torch.sign(torch.randn(V, generator=g))
    x[5] = at * (2 * torch.rand(V, generator=g) - 1)
    return x.clamp(-torch.finfo(dtype).max, torch.finfo(dtype).max).to(dtype)


@pytest.mark.parametrize("cap,scale", [(1e-30, 1.0), (1e-3, 1.0), (0.5, 200.0), (30.0, 1.0), (100.0, 1.0), (128.0, 1.0),
                                       (129.0, 1.0), (3e4, 0.004), (1e10, 1e-9), (500.0, 1.0), (1024.0, 1.0), (1025.0, 1.0), (50.0, 100.0), (3e3, 1.0), (1e4, 1.0),
                                       (3e4, 1.0), (1e5, 1.0), (1e6, 1.0), (1e7, 0.1), (1e20, 1.0), (1e30, 1e-27), (1e37, 1.0)])
@pytest.mark.parametrize("size", [0.0, 0.3, 1.0, 4.0])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
def test_scores_under_a_cap(cap, scale, size, dtype):
    g = torch.Generator().manual_seed(int(size * 10) + 1)
    x = body(cap, size, dtype, g)
    keep = 8
    score, parent, token, _ = (t.cpu() for t in pkg.BeamSelector(1, keep, cap, scale)(x.cuda(), torch.zeros(ROWS, 1, device="cuda")))
    # (the call takes both as fp32; at four caps a cap's relative error enters a difference eight times)
    cap, scale = (float(torch.tensor(v, dtype=torch.float32)) for v in (cap, scale))
    x = x.double()
    top = x.amax(1, keepdim=True)
    # of one sign the difference without cancellation, as sinh(a - b) / (cosh a cosh b)
    a, b = x / cap, top / cap
    u, v = a.abs(), b.abs()
    near = 2 * torch.exp(-2 * torch.minimum(u, v)) * torch.expm1(-2 * (top - x) / cap) / (
        (1 + torch.exp(-2 * u)) * (1 + torch.exp(-2 * v)))
    d = scale * cap * torch.where((a < 0) & (b >= 0), torch.tanh(a) - torch.tanh(b), near)
    want = d - torch.logsumexp(d, 1, keepdim=True)
    order = x.argsort(dim=1, descending=True, stable=True)[:, :keep]
    assert (parent == 0).all()
    # (where the cap saturates in 64 bits, equal scores go by the logit, too)
    assert torch.equal(token, order)
    tol = 2.0 ** -17 * (1 + cap * scale / 8) if cap * scale <= 1024 else 2.0 ** -17 + 2.0 ** -19 * math.log(V)
    best = want.gather(1, order)
    off = (score.double() - best).abs()
    assert (off <= tol + best.abs() * 2.0 ** -23).all(), float((off / (tol + best.abs() * 2.0 ** -23)).max())
    assert (score.diff(dim=1) <= 0).all()
