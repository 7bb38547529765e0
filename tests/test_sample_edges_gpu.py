"""headloss_sample at settings and rows on the edge of what it takes, against the
definition and the 64-bit row reference of test_sample_gpu.py (its tolerances)."""
import math

import numpy as np
import pytest
import torch

import gradient_row_online_gb300 as pkg
from tests.test_sample_gpu import FILTERS, check, noise

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("cap", [0.0, 30.0])
@pytest.mark.parametrize("name", ["own", "k", "kbig", "p", "m", "kp", "kbigp", "pm"])
def test_negative_zero_temperature_is_greedy(name, cap, dtype):
    x, u = noise(6, 4099, dtype, seed=3)
    tok = check(x, u, cap, **dict(FILTERS[name], t=-0.0))
    assert np.array_equal(tok, x.float().argmax(1).cpu().numpy())


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("cap", [0.0, 30.0])
@pytest.mark.parametrize("v", [777, 4099, 128_256])
def test_a_scale_and_temperature_whose_quotient_is_zero(v, cap, dtype):
    """K / T = 0: every token that is not masked weighs the same."""
    x, u = noise(3, v, dtype, seed=v)
    x[1, ::3] = -math.inf
    x[2, v // 4:] = -math.inf
    for f in ({}, dict(p=0.9), dict(p=0.0), dict(k=40, p=0.9), dict(k=700, p=0.5), dict(m=0.5, p=0.7)):
        check(x, u, cap, 1e-30, t=3e38, **f)


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("s,t", [(1e-30, 3e38), (1e-6, 3e38), (0.5, 1.0)])
@pytest.mark.parametrize("v", [777, 4099, 128_256])
def test_capped_rows_with_infinite_logits(v, s, t, dtype):
    """A softcap keeps +inf at a finite z: the largest among other tokens with a mass, at ordinary
    temperatures and at K / T = 0 and just above (where an infinite distance has no bin)."""
    x, u = noise(3, v, dtype, seed=v + 1)
    x[0, v // 2] = math.inf
    x[1, v - 1] = math.inf
    x[1, :v // 2] = -math.inf
    x[2, ::5] = math.inf
    for f in ({}, dict(p=0.9), dict(p=0.0), dict(k=40, p=0.9), dict(k=700, p=0.5), dict(m=0.5, p=0.7)):
        check(x, u, 30.0, s, t=t, **f)


@pytest.mark.parametrize("v", [(1 << 28) - 3, 1 << 28, (1 << 30) + 5])
def test_log_probs_of_rows_past_two_to_the_28_tokens(v):
    x = torch.zeros(1, v, dtype=torch.bfloat16, device="cuda")
    u = torch.tensor([0.625], dtype=torch.float64, device="cuda")
    for t in (None, 0.5):
        tok, lp, dlp, kept = pkg.HeadSampler()(x, u, temperature=t)
        assert int(tok) == math.floor(0.625 * v) and int(kept) == v
        want = -math.log(v)
        assert abs(float(lp) - want) <= 2e-6 + 2e-6 * abs(want)
        assert abs(float(dlp) - want) <= 2e-6 + 2e-6 * abs(want)


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("cap", [30.0, 50.0])
@pytest.mark.parametrize("beside", [0.0, 0.95])
def test_a_dominant_token_of_a_capped_row(beside, cap, dtype):
    """Its log-prob is 0 whatever its logit, in the range of the fit of tanh or past it, alone in its
    word or beside a logit past the fit's range."""
    n, v = 96, 1000
    x, _ = noise(n, v, dtype, seed=1, sigma=0.01)
    x -= 0.5 * cap
    at = torch.arange(n, device="cuda") * 10 + 5
    x[torch.arange(n), at] = (cap * torch.linspace(0.45, 0.9, n, device="cuda")).to(x.dtype)
    if beside:
        x[torch.arange(n), at + 1] = -beside * cap
    u = torch.full((n,), 0.5, dtype=torch.float64, device="cuda")
    for f in ({}, dict(t=0.8, k=40, p=0.9), dict(p=0.9), dict(k=500)):
        assert np.array_equal(check(x, u, cap, **f), at.cpu().numpy())


@pytest.mark.parametrize("dtype,v", [("bf16", 800_003), ("fp16", 1_000_001), ("fp32", 500_009)])
@pytest.mark.parametrize("cap", [0.0, 30.0])
def test_rows_that_are_not_resident(cap, dtype, v):
    """Rows past eight CTAs' shared memory, read from global memory in every pass: ordinary ones,
    few-valued ones, masked ones and +inf, on every way through the kernel."""
    x, u = noise(6, v, dtype, seed=v, sigma=2.0, pitch=v + 3)
    x[1] = (x[1].float() / 2).round().to(x.dtype)  # a few values
    x[2, ::3] = -math.inf
    x[2, 1::7] = math.nan
    x[3, [5, v // 2, v - 1]] = math.inf
    x[4] = -math.inf
    x[5, :v - 9] = -math.inf
    for f in ({}, dict(t=0.7, k=40, p=0.9), dict(p=0.9), dict(p=0.3, m=0.2), dict(k=5000), dict(k=3000, p=0.9),
              dict(t=0.0), dict(m=0.05)):
        tok = check(x, u, cap, **f)
        assert tok[4] == -1 and tok[5] >= v - 9
        assert cap or tok[3] in (5, v // 2, v - 1)
