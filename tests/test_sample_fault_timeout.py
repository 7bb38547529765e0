"""The sampling kernel's bounded copy waits, without a GPU fault.

A test-only build of the library (-DHL_FAULT_INJECT) leaves out the copies of one row and
shortens the waits.  That row has no token and error bit 1 is set; the other rows, and the next
call, are as ever.  No barrier whose copy was left out is used again, and every wait is bounded.
"""
import ctypes

import pytest
import torch

import gradient_row_online_gb300 as pkg
from gradient_row_online_gb300 import build as B
from gradient_row_online_gb300 import headloss as hlb
from tests.test_sample_gpu import noise

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("settings", [{}, dict(top_p=0.9), dict(top_k=40, top_p=0.9)])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("v", [1031, 128_256])
def test_a_lost_copy_gives_up_its_row_alone(v, dtype, settings):
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    n, drop = 5, 3
    x, u = noise(n, v, dtype, seed=v)
    want = pkg.HeadSampler()(x, u, **settings)
    lib = ctypes.CDLL(B.build(fault_inject=True))
    lib.headloss_sample.argtypes = hlb.load_library().headloss_sample.argtypes
    lib.headloss_sample_test_inject.argtypes = [ctypes.c_int64, ctypes.c_ulonglong]
    lib.headloss_sample_test_inject.restype = None
    sampler = pkg.HeadSampler()
    sampler._call = lib.headloss_sample
    lib.headloss_sample_test_inject(drop, 20_000_000)  # 20 ms
    got = sampler(x, u, **settings)
    assert sampler.device_error() == 2
    rest = [i for i in range(n) if i != drop]
    assert all(torch.equal(a[rest], b[rest]) for a, b in zip(want, got))
    assert [float(a[drop]) for a in got] == [-1.0, 0.0, 0.0, 0.0]
    lib.headloss_sample_test_inject(-1, 0)
    got = sampler(x, u, **settings)
    assert sampler.device_error() == 0
    assert all(torch.equal(a, b) for a, b in zip(want, got))
