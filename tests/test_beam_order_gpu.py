"""The order between beams where the scores' difference is less than fp32 shows: as fp64 has it.

Rows of two allowed tokens with logits a and 0: the better one's log-prob is -log(1 + e^-a). The row's sum is held in fp32
and its exponentials are off by 2^-22: 4e-7 of a log-prob at most, where the beams differ by 1e-5."""
import math

import numpy as np
import pytest
import torch

import gradient_row_online_gb300 as pkg

pytestmark = pytest.mark.gpu


def pair(a1, before):
    """Scores and leading logits of two beams, the second better by 1e-5 but not as fp32 adds it up."""
    s1 = np.float32(before)
    s0 = np.nextafter(s1, np.float32(-np.inf))
    lp1 = -math.log1p(math.exp(-a1))
    lp0 = lp1 + (float(s1) - float(s0)) - 1e-5
    a0 = float(np.float32(-math.log(math.expm1(-lp0))))
    lp0 = -math.log1p(math.exp(-a0))
    assert 0.9e-5 < (float(s1) + lp1) - (float(s0) + lp0) < 1.1e-5
    return (s0, s1), (a0, a1), np.float32(s0 + np.float32(lp0)) >= np.float32(s1 + np.float32(lp1))


@pytest.mark.parametrize("before", [-1e4, -3e4, -1e5])
@pytest.mark.parametrize("V", [2, 1000, 40000])
def test_a_difference_that_fp32_hides(before, V):
    hidden = 0
    for a1 in (0.3, 0.5, 1.0, 1.25, 1.5):
        s, a, other = pair(float(np.float32(a1)), before)
        hidden += other
        x = torch.full((4, V), -math.inf)
        x[:, 0] = 0.0
        x[0, V - 1], x[1, V - 1], x[2, V - 1], x[3, V - 1] = a[0], a[1], a[1], a[0]
        scores = torch.tensor([[s[0], s[1]], [s[1], s[0]]])
        _, p, t, _ = pkg.BeamSelector(2)(x.cuda(), scores.cuda())
        assert p.tolist() == [[1, 0], [0, 1]] and (t == V - 1).all(), a1
    assert hidden >= 3  # fp32 alone would have left the first beam in front
