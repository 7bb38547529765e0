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
