"""A beam search's selection where a CTA goes over many batches of a row: few CTAs a row, long rows, and
rows whose order, masks or values are at their most awkward.  Tolerance as in test_beam_gpu, with twice
as many additions a thread for each doubling of a slice's batches (up to eight here): 2^-14."""
import math

import pytest
import torch

import gradient_row_online_gb300 as pkg

pytestmark = pytest.mark.gpu

ROWS = 960  # enough that a row is one CTA's


def expected(x, keep, cap, scale):
    """Of rows that are requests of their own: the keep best tokens and their log-probs."""
    x = torch.where(x.isnan(), -math.inf, x.double())
    top, token = x.sort(dim=1, descending=True, stable=True)
    top, token = top[:, :keep], token[:, :keep]
    z = cap * torch.tanh(x / cap) if cap else x
    zt = cap * torch.tanh(top / cap) if cap else top
    best = zt[:, :1]
    d = torch.where(x == -math.inf, -math.inf, torch.where(z == best, 0.0, (z - best) * scale))
    lse = torch.log(torch.exp(d).sum(1, keepdim=True))
    s = torch.where(zt == best, 0.0, (zt - best) * scale) - lse
    none = (top == -math.inf) | (s == -math.inf)
    return torch.where(none, -math.inf, s), torch.where(none, -1, token)


def rows(kind, V, dtype, g):
    x = 3 * torch.randn(ROWS, V, generator=g, device="cuda")
    if kind == "rising":
        x = x.sort(dim=1).values
    elif kind == "falling":
        x = x.sort(dim=1, descending=True).values
    elif kind == "lowest first":  # masked by the type's lowest value, most of all at the front
        x[:, :V * 2 // 3] = torch.finfo(dtype).min
    elif kind == "nothing first":
        x[:, :V * 2 // 3] = -math.inf
    elif kind == "few allowed":
        x.masked_fill_(torch.rand(ROWS, V, generator=g, device="cuda") < 0.9997, -math.inf)
    elif kind == "equal":
        x = torch.full_like(x, 0.5)
    elif kind == "two values":
        x = (x > 0).float()
    elif kind == "steps":  # far above the first batch, and again
        x[:, V // 3:] += 150.0
        x[:, 2 * V // 3:] += 300.0
    elif kind == "nan":
        x.masked_fill_(torch.rand(ROWS, V, generator=g, device="cuda") < 0.001, math.nan)
        x[:, :20000] = math.nan
    elif kind == "infinity":
        x[::2, V - 7] = math.inf
        x[::3, 11] = math.inf
    elif kind == "wide":
        x *= 1e4
    return x.to(dtype)


KINDS = ["random", "rising", "falling", "lowest first", "nothing first", "few allowed", "equal", "two values", "steps",
         "nan", "infinity", "wide"]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("cap,scale", [(0.0, 1.0), (30.0, 0.5)])
def test_long_rows(kind, dtype, cap, scale):
    V = 60001 if dtype is not torch.float32 else 30001  # four batches, off the 16-byte grid
    g = torch.Generator("cuda").manual_seed(len(kind))
    x = rows(kind, V, dtype, g)
    before = torch.zeros(ROWS, 1, device="cuda")
    for keep in (1, 16, 40):
        score, parent, token, _ = pkg.BeamSelector(1, keep, cap, scale)(x, before)
        want, at = expected(x, keep, cap, scale)
        if cap == 0 or kind not in ("wide", "steps", "infinity"):
            assert torch.equal(token, at)
        # (where the cap saturates in 64 bits, equal scores go by the logit, as these do, too)
        assert torch.equal(token.sort(1).values, at.sort(1).values)
        assert torch.equal(parent, torch.where(at < 0, -1, 0).int())
        fine = at >= 0
        off = (score.double() - want)[fine].abs()
        assert (off <= 2.0 ** -14 * (1 + cap * scale / 8) + want[fine].abs() * 2.0 ** -23).all(), float(off.max())
        again = pkg.BeamSelector(1, keep, cap, scale)(x, before)
        assert all(torch.equal(a, b) for a, b in zip(again, (score, parent, token)))


def test_rows_far_apart():
    """Rows whose offsets pass 32 bits."""
    V, ld = 5000, 1 << 30
    buf = torch.zeros(3 * ld + V, dtype=torch.bfloat16, device="cuda")
    x = buf.as_strided((4, V), (ld, 1))
    g = torch.Generator("cuda").manual_seed(1)
    x.copy_(torch.randn(4, V, generator=g, device="cuda"))
    sel = pkg.BeamSelector(4, 8)
    s = torch.zeros(1, 4, device="cuda")
    for a, b in zip(sel(x, s), sel(x.contiguous(), s)):
        assert torch.equal(a, b)


def test_reorder_beyond_32_bits():
    n = (1 << 30) + (1 << 20)
    state = torch.zeros(4, n, dtype=torch.int8, device="cuda")
    for r in range(4):
        state[r, -4096:] = r + 1
        state[r, :4096] = 10 + r
    parents = torch.tensor([[3, 2, 2, 0]], dtype=torch.int32, device="cuda")
    pkg.StateReorder([state], 4)(parents)
    assert state[:, -1].tolist() == [4, 3, 3, 1] and state[:, 0].tolist() == [13, 12, 12, 10]
    assert state[:, -4096:].eq(state[:, -1:]).all() and state[:, 4096:-4096].eq(0).all()
    cache = state.view(4, 2, -1, 128)  # as (rows, heads, positions, width)
    begin = torch.tensor([cache.shape[2] - 2], dtype=torch.int32, device="cuda")
    pkg.StateReorder([cache], 4, axis=2)(torch.tensor([[1, 0, 3, 2]], dtype=torch.int32, device="cuda"), begin, begin + 9)
    assert state[:, -1].tolist() == [3, 4, 1, 3] and state[:, 0].tolist() == [13, 12, 12, 10]
