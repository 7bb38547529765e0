"""headloss_clip_grads where test_clip_gpu.py does not go: subnormal gradients, lists through the
workspace, calls that none waits for.  Tolerances are those of test_clip_gpu.py, and
beside them half a step of fp32's subnormals (2^-150) for a norm that is rounded to them."""
import math

import pytest
import torch

import gradient_row_online_gb300 as pkg
from tests.test_clip_gpu import STEP, TINY, check, make

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


def many(n, dtypes, seed=0, flat=False):
    """n small tensors of mixed sizes, some of them empty, and one that spans many tiles."""
    sizes = [(37 * i) % 301 for i in range(n)]
    sizes[n // 3] = 50_001
    return make(sizes, dtypes, seed=seed, flat=flat)


@pytest.mark.parametrize("n", [16, 17, 64, 65, 160, 161, 320, 321, 512, 513, 960, 961, 1024, 1025, 1537, 3000])
def test_lists_of_every_length(n):
    """Each size of the list in kernel arguments and lists through the workspace, to their ends
    (`n` counts the tensors with elements)."""
    for dtypes, flat in ((("bf16", "fp32", "fp16"), False), (("bf16",), True)):
        grads = many(n, dtypes, seed=n, flat=flat)
        empty = sum(g.numel() == 0 for g in grads)
        grads += make([5] * empty, dtypes, seed=1)
        assert sum(g.numel() > 0 for g in grads) == n
        check(grads, 0.37)
        check(grads, 0.37, 0.5, inplace=True)


def test_calls_of_one_handle_that_none_waits_for():
    """Lists of other lengths and grids one after the other on a stream that is still busy: all are
    enqueued before the first runs."""
    sets = [many(1100, ("bf16",), seed=1), make([3_000_000, 5], ("fp32",), seed=2), make([9], ("fp16",), seed=3),
            many(2500, ("fp32", "bf16"), seed=4), make([20_000_000], ("bf16",), seed=5),
            make([4000] * 300, ("bf16",), seed=6), many(961, ("fp16",), seed=7)]
    norms = [math.sqrt(sum(float(g.double().square().sum()) for g in grads)) for grads in sets]
    clipper = pkg.GradClipper([], max_grads=3000)
    outs = [[[torch.empty_like(g) for g in grads] for grads in sets] for _ in range(3)]
    got = []
    torch.cuda.synchronize()
    torch.cuda._sleep(400_000_000)
    for turn in outs:
        for grads, out in zip(sets, turn):
            clipper.bind(grads, out)
            got.append(clipper(1.0))
    torch.cuda.synchronize()
    for stats, (grads, out, want) in zip(got, [(g, o, w) for turn in outs
                                               for g, o, w in zip(sets, turn, norms)]):
        norm, factor = stats.tolist()
        assert abs(norm - want) <= 2.0 ** -16 * want and abs(factor - 1 / want) <= 2.0 ** -15 * factor
        for g, o in zip(grads, out):
            ref = g.double() / want
            assert bool(((o.double() - ref).abs() <= STEP[g.dtype] * ref.abs() + TINY[g.dtype]).all())
