"""A beam search's selection under a cap where a batch's candidates are listed a second time (a row that rises by more
than a list holds): what the list takes off the sum is what was added.

One token has all of a row's mass: the others lie 64 octaves and more below. The sum is then its exponential, from the
fit of tanh or from its other form (at a cap of 1000 up to 2^-21 * 1000 = 5e-4 off), less the same, plus 1: the score is
0 but for that addition (2^-24), the fixed point (2^-40) and the logarithm's rounding."""
import pytest
import torch

import gradient_row_online_gb300 as pkg

pytestmark = pytest.mark.gpu

ROWS = 960  # a row is one CTA's


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("cap", [300.0, 1000.0])
@pytest.mark.parametrize("at", [0.3, 0.7, 0.95])  # within the fit's range, and beyond
@pytest.mark.parametrize("keep", [1, 16, 40])
def test_a_token_with_all_the_mass(dtype, cap, at, keep):
    batch = 2048 * (4 if dtype is torch.float32 else 8)
    V = 2 * batch + 77
    g = torch.Generator("cuda").manual_seed(keep)
    x = 0.1 * cap * torch.rand(ROWS, V, generator=g, device="cuda") - 0.6 * cap
    x[:, batch:] += 0.2 * cap
    top = torch.randint(batch, V, (ROWS, 1), generator=g, device="cuda")
    x.scatter_(1, top, cap * at * (0.9 + 0.1 * torch.rand(ROWS, 1, generator=g, device="cuda")))
    score, _, token, _ = pkg.BeamSelector(1, keep, cap)(x.to(dtype), torch.zeros(ROWS, 1, device="cuda"))
    assert torch.equal(token[:, :1], top)
    assert float(score[:, 0].abs().max()) <= 2.0 ** -22, float(score[:, 0].abs().max())
