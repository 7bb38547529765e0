"""headloss_clip_grads against the formula in 64 bits.

norm: fp32 squares (2^-24 relative each), sums of at most a few hundred of them
in fp32 and fp64 beyond: within 2^-16 relative (a sum of n positive terms errs by
at most n 2^-24, n <= 256), and the rounding to fp32.  Outputs: the factor carries
the norm's error and one rounding, the product one more; the result is one step
of the output type around the exact product, so it is held to 1 ulp of the type
beside 2^-15 relative for fp32 (where the factor's error is above the type's)."""
import math

import numpy as np
import pytest
import torch

import gradient_row_online_gb300 as pkg
from gradient_row_online_gb300 import headloss as hlb

pytestmark = pytest.mark.gpu

DT = {"fp32": torch.float32, "bf16": torch.bfloat16, "fp16": torch.float16}
STEP = {torch.float32: 2.0 ** -15, torch.bfloat16: 2.0 ** -7, torch.float16: 2.0 ** -9}
TINY = {torch.float32: 1e-44, torch.bfloat16: 2e-40, torch.float16: 1.2e-7}


def make(sizes, dtypes, seed=0, sigma=1.0, flat=False):
    g = torch.Generator("cuda").manual_seed(seed)
    out = []
    for i, n in enumerate(sizes):
        out.append((torch.randn(n, generator=g, device="cuda") * sigma).to(DT[dtypes[i % len(dtypes)]]))
    if flat:  # views of one buffer, off the 16-byte grid
        whole = torch.cat(out)
        out = list(whole.split(list(sizes)))
    return out


def check(grads, max_norm, inv_scale=1.0, inplace=False):
    want = math.sqrt(sum(float(g.double().square().sum()) for g in grads)) * inv_scale
    factor = inv_scale * (max_norm / want if want > max_norm else 1.0)
    before = [g.double() for g in grads]
    if inplace:
        outs = grads
        clipper = pkg.GradClipper(grads)
    else:
        whole = [torch.full((g.numel() + 2,), 7.0, dtype=g.dtype, device="cuda") for g in grads]
        outs = [w[1:-1] for w in whole]
        clipper = pkg.GradClipper(grads, outs)
    stats = clipper(max_norm, inv_scale).cpu().numpy()
    assert abs(stats[0] - want) <= 2.0 ** -16 * want, (stats, want)
    assert abs(stats[1] - factor) <= 2.0 ** -15 * factor, (stats, factor)
    for g, o, b in zip(grads, outs, before):
        ref = b * factor
        off = (o.double() - ref).abs()
        assert bool((off <= STEP[g.dtype] * ref.abs() + TINY[g.dtype]).all())
        if not inplace:
            assert torch.equal(g.double(), b)
    if not inplace:
        for w in whole:
            assert float(w[0]) == 7.0 and float(w[-1]) == 7.0
    return stats, outs


SIZES = {"one": [1], "few": [3, 1, 8, 7], "odd": [1, 33, 1000, 16383, 16384, 16385, 4097, 5],
         "long": [3_000_001, 17, 70_000], "many": [257 + 3 * (i % 11) for i in range(700)],
         "big": [40_000_003, 1_000_000]}


@pytest.mark.parametrize("name", SIZES)
@pytest.mark.parametrize("dtypes", [("fp32",), ("bf16",), ("fp16",), ("bf16", "fp32", "fp16")])
def test_norm_and_clip(name, dtypes):
    grads = make(SIZES[name], dtypes, seed=len(name))
    check(grads, 0.37)
    check(grads, 1e9)
    check(grads, 0.37, inplace=True)


@pytest.mark.parametrize("dtype", ["fp32", "bf16", "fp16"])
def test_views_off_the_grid(dtype):
    grads = make([5, 1001, 3, 70_001, 16_384, 9], (dtype,), flat=True)
    check(grads, 2.0, 0.25)
    check(grads, 2.0, inplace=True)


def test_in_place_without_clipping_keeps_every_bit():
    grads = make([1000, 70_001], ("bf16", "fp32"), sigma=1e-3)
    bits = [g.clone() for g in grads]
    stats, _ = check(grads, 1e4, inplace=True)
    assert stats[1] == 1.0
    assert all(torch.equal(a, b) for a, b in zip(bits, grads))


def test_inv_scale():
    grads = make([4096, 33], ("fp16", "fp32"), sigma=512.0)
    check(grads, 1.0, 1.0 / 1024)
    check(grads, 1e6, 1.0 / 1024)
    check(grads, 1e6, 1.0 / 1024, inplace=True)


@pytest.mark.parametrize("sigma", [1e-37, 1e-30, 1e-21, 1e-12, 1e12, 1e17, 1e25, 1e33])
@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
def test_the_types_range(sigma, dtype):
    """Squares far below and far above fp32's range."""
    grads = make([20_000, 3], (dtype,), sigma=sigma)
    check(grads, sigma * 3)
    check(grads + make([5000], (dtype,), sigma=1.0), 0.5 + sigma)


def test_zero_gradients():
    grads = [torch.zeros(50_000, device="cuda", dtype=torch.bfloat16), torch.zeros(3, device="cuda")]
    stats, _ = check(grads, 1.0)
    assert stats[0] == 0 and stats[1] == 1


@pytest.mark.parametrize("bad", [math.inf, -math.inf, math.nan])
def test_a_norm_that_is_not_finite_leaves_the_values(bad):
    for dtype in DT:
        grads = make([30_000, 1000], (dtype,))
        grads[1][77] = bad
        outs = [torch.empty_like(g) for g in grads]
        stats = pkg.GradClipper(grads, outs)(1.0, 0.5).cpu().numpy()
        assert not np.isfinite(stats[0]) and stats[1] == 0.5
        assert torch.equal(outs[0], (grads[0].float() * 0.5).to(grads[0].dtype))
        same = (grads[1].float() * 0.5).to(grads[1].dtype)
        assert torch.equal(outs[1].nan_to_num(5.0), same.nan_to_num(5.0))


def test_empty_tensors_and_an_empty_list():
    grads = make([5, 100], ("fp32",))
    empty = torch.empty(0, device="cuda")
    check([empty, grads[0], empty, grads[1], empty], 0.1)
    stats = pkg.GradClipper([])(1.0).cpu().numpy()
    assert stats[0] == 0 and stats[1] == 1


def test_the_same_bits_every_time_and_on_another_stream():
    grads = make([3_000_001, 70_000, 5], ("bf16", "fp32"))
    outs = [torch.empty_like(g) for g in grads]
    clipper = pkg.GradClipper(grads, outs)
    first = clipper(0.5).clone()
    kept = [o.clone() for o in outs]
    side = torch.cuda.Stream()
    for _ in range(5):
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            again = clipper(0.5)
        torch.cuda.current_stream().wait_stream(side)
        assert torch.equal(first, again)
        assert all(torch.equal(a, b) for a, b in zip(kept, outs))


def test_binding_other_tensors():
    clipper = pkg.GradClipper(make([10, 20], ("fp32",)), max_grads=3)
    grads = make([700, 3, 9000], ("bf16",), seed=3)
    outs = [torch.empty_like(g) for g in grads]
    clipper.bind(grads, outs)
    want = math.sqrt(sum(float(g.double().square().sum()) for g in grads))
    assert abs(float(clipper(1.0)[0]) - want) <= 2.0 ** -16 * want
    with pytest.raises(ValueError):
        clipper.bind(make([1, 1, 1, 1], ("fp32",)))


def test_back_to_back_calls_of_one_handle():
    """Lists of other sizes one after the other on a stream, none waited for."""
    clipper = pkg.GradClipper(make([10], ("fp32",)), max_grads=400)
    sets = [make([4000] * 300, ("bf16",), seed=1), make([3_000_000, 5], ("fp32",), seed=2),
            make([9], ("fp16",), seed=3), make([20_000_000], ("bf16",), seed=4)]
    got, want = [], []
    for _ in range(3):
        for grads in sets:
            clipper.bind(grads, [torch.empty_like(g) for g in grads])
            got.append(clipper(1.0))
            want.append(math.sqrt(sum(float(g.double().square().sum()) for g in grads)))
    for a, b in zip(got, want):
        assert abs(float(a[0]) - b) <= 2.0 ** -16 * b


def test_graph_capture():
    grads = make([5000, 33, 900_000], ("bf16", "fp32"))
    outs = [torch.zeros_like(g) for g in grads]
    clipper = pkg.GradClipper(grads, outs)
    want = clipper(0.5).clone()
    kept = [o.clone() for o in outs]
    stats = torch.zeros(2, device="cuda")
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        clipper(0.5, stats=stats)
    for o in outs:
        o.zero_()
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(stats, want) and all(torch.equal(a, b) for a, b in zip(kept, outs))


def test_offsets_past_two_to_the_31():
    n = (1 << 31) + 4097
    g = torch.zeros(n, dtype=torch.bfloat16, device="cuda")
    g[-5:] = 3.0
    g[:2] = 4.0
    pkg.GradClipper([g])(1.0)
    norm = math.sqrt(5 * 9.0 + 2 * 16.0)
    assert torch.allclose(g[-5:].float(), torch.full((5,), 3.0 / norm, device="cuda"), rtol=2.0 ** -8)
    assert torch.allclose(g[:2].float(), torch.full((2,), 4.0 / norm, device="cuda"), rtol=2.0 ** -8)


def test_refusals():
    x = make([8], ("fp32",))
    clipper = pkg.GradClipper(x)
    for args in ((0.0,), (-1.0,), (math.nan,), (1.0, 0.0), (1.0, math.inf), (1.0, math.nan)):
        with pytest.raises(hlb.HeadlossError):
            clipper(*args)
    with pytest.raises(ValueError):
        pkg.GradClipper(x, [])
    with pytest.raises(ValueError):
        pkg.GradClipper(x, [x[0].bfloat16()])
    with pytest.raises(ValueError):
        pkg.GradClipper([torch.zeros(4, 4, device="cuda").t()[1:]])
    with pytest.raises(ValueError):
        pkg.GradClipper([torch.zeros(4)])
