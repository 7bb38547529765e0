"""The operators behind the head together: beam search steps (8-bit logits, selection, reordering), and a
training step (8-bit logits, the loss, both gradients, clipping)."""
import pytest
import torch

import gradient_row_online_gb300 as pkg
from gradient_row_online_gb300 import headloss as hl

pytestmark = pytest.mark.gpu


def test_beam_steps_keep_beams_and_states_together():
    from examples.beam_step import Decoder
    R, B, steps, prompt = 3, 4, 6, 5
    d = Decoder(R, B, 256, 4, prompt, steps, 2000, eos=7)
    prompt_cache = torch.randn(R, 4, prompt, 64, device="cuda").bfloat16()
    d.cache[:, :, :prompt] = prompt_cache.repeat_interleave(B, 0)
    states = [d.state.clone()]
    history = None
    for t in range(steps):
        before, caches = d.state.clone(), d.cache.clone()
        scores, ended = d.scores.clone(), d.ended.clone()
        logits = d.head.logits(before)
        parents, tokens = d.step()
        # the selection's scores are the parents' plus the token's log-prob
        lp = torch.log_softmax(logits.double(), 1).view(R, B, -1)
        p = parents.long()
        assert (p >= 0).all()
        want = scores.double().gather(1, p) + torch.where(ended.gather(1, p), 0.0, lp[torch.arange(R)[:, None].cuda(), p, tokens])
        assert ((d.scores.double() - want).abs() <= 2.0 ** -16 + want.abs() * 2.0 ** -23).all()
        # the states that the step went on from are the parents'
        rows = (torch.arange(R, device="cuda")[:, None] * B + p).view(-1)
        new = torch.tanh(before[rows] @ d.mix + d.embedding[tokens.view(-1)])
        assert torch.equal(d.state, new)
        at = prompt + t
        assert torch.equal(d.cache[:, :, prompt:at], caches[rows][:, :, prompt:at])
        assert torch.equal(d.cache[:, :, :prompt], caches[:, :, :prompt])
        history = tokens[..., None] if history is None else torch.cat(
            (torch.take_along_dim(history, p[..., None], 1), tokens[..., None]), 2)
    assert len({tuple(h) for h in history[0].tolist()}) == B  # beams are different sequences
    assert d.head.device_error() == 0 and len(states) == 1


@pytest.mark.parametrize("N,D,V", [(70, 256, 1000), (200, 520, 4001)])
def test_training_step_through_the_8_bit_head(N, D, V):
    """Gradients of cross-entropy through the head against those of 64-bit logits from the same 8-bit weights and
    hidden states; the loss's gradient is quantised once more (1 x 128, e4m3: half a step is 2^-4 of a value, or
    2^-10 of the block's largest), and so are the hidden states over the tokens."""
    g = torch.Generator("cuda").manual_seed(N)
    w = torch.randn(V, D, generator=g, device="cuda") * D ** -0.5
    x = torch.randn(N, D, generator=g, device="cuda")
    y = torch.randint(V, (N,), generator=g, device="cuda")
    head = pkg.Fp8Head(w, train=True)
    loss = pkg.HeadLoss(hl.HEADLOSS_CE, hl.make_weights(ce=1.0))
    logits = head.logits(x)
    grad = torch.empty_like(logits)
    scalars = loss(logits, y, grad_out=grad)
    gx, gw = head.backward(grad, x)
    clipper = pkg.GradClipper([gw])
    norm = clipper(1e9)
    codes = head.q[:, :D].view(torch.float8_e4m3fn).double()
    wide = head.scales.double().repeat_interleave(128, 0)[:V].repeat_interleave(128, 1)[:, :D]
    w8 = codes * wide
    p = torch.softmax(logits.double(), 1)
    assert abs(float(scalars[1]) - float(-torch.log(p[torch.arange(N), y]).mean())) <= 1e-5 * float(scalars[1])
    dl = p.clone()
    dl[torch.arange(N), y] -= 1
    dl /= N

    def block(t, rows):  # the largest magnitude of each element's block
        n, k = t.shape
        u = torch.nn.functional.pad(t.abs(), (0, -k % 128, 0, -n % rows)).view(-(-n // rows), rows, -(-k // 128), 128)
        m = u.amax((1, 3))
        return m.repeat_interleave(rows, 0)[:n].repeat_interleave(128, 1)[:, :k]
    # |error| of a product <= sum of |a's error| |b| + |a| |b's error| + both; fp32 sums are far below
    da = dl.abs() * 2.0 ** -4 + block(dl, 1) * 2.0 ** -10
    assert ((gx.double() - dl @ w8).abs() <= (da @ w8.abs()) * 1.01 + 1e-12).all()
    dt = dl.t().contiguous()
    dat = dt.abs() * 2.0 ** -4 + block(dt, 1) * 2.0 ** -10
    xt = x.double().t().contiguous()
    dxt = xt.abs() * 2.0 ** -4 + block(xt, 128) * 2.0 ** -10
    bound = dat @ xt.abs().t() + dt.abs() @ dxt.t() + dat @ dxt.t()
    assert ((gw.double() - dt @ xt.t()).abs() <= bound * 1.01 + 1e-12).all()
    assert abs(float(norm[0]) - float(gw.double().norm())) <= 1e-5 * float(norm[0])
    assert head.device_error() == 0


def test_gradients_against_differences():
    """A step against the gradient lowers the loss of the unquantised head by about its square, within the
    relative error of 8-bit gradients (each factor's values are off by 2^-4 at most)."""
    g = torch.Generator("cuda").manual_seed(3)
    N, D, V = 96, 256, 700
    w = torch.randn(V, D, generator=g, device="cuda") * D ** -0.5
    x = torch.randn(N, D, generator=g, device="cuda")
    y = torch.randint(V, (N,), generator=g, device="cuda")
    head = pkg.Fp8Head(w, train=True)
    logits = head.logits(x)
    grad = torch.empty_like(logits)
    pkg.HeadLoss(hl.HEADLOSS_CE, hl.make_weights(ce=1.0))(logits, y, grad_out=grad)
    gx, gw = (t.double() for t in head.backward(grad, x))

    def ce(x64, w64):
        return float(torch.nn.functional.cross_entropy(x64 @ w64.t(), y))
    x64, w64, h = x.double(), w.double(), 1e-4
    for dx, dw in ((gx, torch.zeros_like(gw)), (torch.zeros_like(gx), gw)):
        size = float((dx.square().sum() + dw.square().sum()))
        unit = h / size ** 0.5
        slope = (ce(x64 + unit * dx, w64 + unit * dw) - ce(x64 - unit * dx, w64 - unit * dw)) / (2 * unit)
        assert abs(slope / size - 1) <= 2 * 2.0 ** -4 + 2.0 ** -8
