"""headloss_clip_grads where test_clip_gpu.py does not go: subnormal gradients, lists through the
workspace, calls that none waits for.  Tolerances are those of test_clip_gpu.py, and
beside them half a step of fp32's subnormals (2^-150) for a norm that is rounded to them."""
import math

import pytest
import torch

import gradient_row_online_gb300 as pkg
from tests.test_clip_gpu import STEP, TINY, make

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("sigma", [1e-38, 1e-39, 1e-40, 1e-41, 1e-43, 1e-44])
def test_subnormal_gradients(sigma, dtype):
    for sizes in ([64], [20_000, 3], [70_001] * 5):
        grads = make(sizes, (dtype,), sigma=sigma, seed=sizes[0])
        want = math.sqrt(sum(float(g.double().square().sum()) for g in grads))
        # a limit that fp32 holds, about half the norm
        limit = float(torch.tensor(max(want / 2, 2.0 ** -149), dtype=torch.float32))
        factor = limit / want if want > limit else 1.0
        outs = [torch.empty_like(g) for g in grads]
        stats = pkg.GradClipper(grads, outs)(limit).tolist()
        assert abs(stats[0] - want) <= 2.0 ** -16 * want + 2.0 ** -150, (stats, want)
        assert abs(stats[1] - factor) <= 2.0 ** -15 * factor, (stats, factor)
        for g, o in zip(grads, outs):
            ref = g.double() * factor
            assert bool(((o.double() - ref).abs() <= STEP[g.dtype] * ref.abs() + TINY[g.dtype]).all())


def test_the_least_subnormal_alone():
    g = torch.zeros(5000, device="cuda")
    g[4321] = 2.0 ** -149
    assert pkg.GradClipper([g])(1.0).tolist() == [2.0 ** -149, 1.0]
