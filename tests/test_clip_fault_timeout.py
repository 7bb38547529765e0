"""The clipping kernel's bounded barrier, without a GPU fault.

A test-only build of the library (-DHL_FAULT_INJECT) lets one CTA come late to the grid's
barrier and shortens the others' wait.  All CTAs then take one outcome: nothing is written and
both stats are NaN, although the late CTA arrives in the end; the handle's next call is an
ordinary one.  Every wait is bounded.
"""
import ctypes
import math

import pytest
import torch

from gradient_row_online_gb300 import build as B
from gradient_row_online_gb300 import headloss as hlb

pytestmark = pytest.mark.gpu


def _fault_lib():
    lib = ctypes.CDLL(B.build(fault_inject=True))
    vp, i32, u64 = ctypes.c_void_p, ctypes.c_int, ctypes.c_ulonglong
    lib.headloss_clip_create.argtypes = [i32, ctypes.POINTER(vp)]
    lib.headloss_clip_grads.argtypes = [vp, ctypes.POINTER(hlb.headloss_gradient), i32, ctypes.c_float,
                                        ctypes.c_float, vp, vp]
    lib.headloss_clip_destroy.argtypes = [vp]
    lib.headloss_clip_destroy.restype = None
    lib.headloss_clip_test_inject.argtypes = [vp, i32, u64, u64]
    lib.headloss_clip_test_inject.restype = None
    return lib


@pytest.mark.parametrize("inplace", [False, True])
@pytest.mark.parametrize("late", [0, 7, 150])
def test_a_late_cta_fails_the_whole_call(late, inplace):
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    lib = _fault_lib()
    n = 4_000_000  # fp32: more than 150 CTAs, a tile or more a warp
    g = torch.randn(n, device="cuda", generator=torch.Generator("cuda").manual_seed(1))
    kept = g.clone()
    out = g if inplace else torch.full_like(g, 7.0)
    before = out.clone()
    stats = torch.zeros(2, device="cuda")
    entry = (hlb.headloss_gradient * 1)()
    entry[0].grad, entry[0].out, entry[0].n, entry[0].dtype = g.data_ptr(), out.data_ptr(), n, 0
    h = ctypes.c_void_p()
    assert lib.headloss_clip_create(1, ctypes.byref(h)) == 0
    stream = torch.cuda.current_stream().cuda_stream

    def call():
        assert lib.headloss_clip_grads(h, entry, 1, 1.0, 0.5, stats.data_ptr(), stream) == 0
        torch.cuda.synchronize()
        return stats.tolist()

    for _ in range(2):
        # 100 ms late where the others wait for 10 ms
        lib.headloss_clip_test_inject(h, late, 100_000_000, 10_000_000)
        norm, factor = call()
        assert math.isnan(norm) and math.isnan(factor)
        assert torch.equal(out, before) and torch.equal(g, kept)
    # 10 ms late where the others wait for 2 s
    lib.headloss_clip_test_inject(h, late, 10_000_000, 0)
    want = 0.5 * float(kept.double().square().sum().sqrt())
    norm, factor = call()
    assert abs(norm - want) <= 2.0 ** -16 * want and abs(factor - 0.5 / want) <= 2.0 ** -15 * factor
    assert torch.allclose(out.double(), kept.double() * (0.5 / want), rtol=2.0 ** -15, atol=1e-44)
    lib.headloss_clip_destroy(h)
