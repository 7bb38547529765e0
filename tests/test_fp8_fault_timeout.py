"""The 8-bit product's bounded waits, without a GPU fault.

A test-only build of the library (-DHL_FAULT_INJECT) leaves out one copy of the first CTA and shortens
the waits: that CTA's roles give up, bit 0 of the error word is set, the other tiles and the next call are
as ever.  No barrier whose copy was left out is used again."""
import ctypes

import pytest
import torch

import gradient_row_online_gb300 as pkg
from gradient_row_online_gb300 import build as B
from gradient_row_online_gb300 import headloss as hlb

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("tokens", [3, 200])
@pytest.mark.parametrize("drop", [0, 2, 7])
def test_a_lost_copy_sets_the_error_word(tokens, drop):
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    g = torch.Generator().manual_seed(tokens + drop)
    head = pkg.Fp8Head(torch.randn(1500, 1024, generator=g).cuda())
    x = torch.randn(tokens, 1024, generator=g).cuda()
    want = head.logits(x)
    lib = ctypes.CDLL(B.build(fault_inject=True))
    own = hlb.load_library()
    lib.headloss_fp8_linear.argtypes = own.headloss_fp8_linear.argtypes
    lib.headloss_fp8_test_inject.argtypes = [ctypes.c_int, ctypes.c_ulonglong]

    class Faulty:
        headloss_fp8_linear = lib.headloss_fp8_linear
        headloss_fp8_linear_workspace = own.headloss_fp8_linear_workspace
    head._lib = Faulty
    torch.cuda.synchronize()
    assert lib.headloss_fp8_test_inject(drop, 5_000_000) == 0  # 5 ms
    got = head.logits(x)
    assert head.device_error() == 1 and head.device_error() == 0
    assert torch.equal(got[:, 256:], want[:, 256:]) or tokens > 128  # (the first tile is the first CTA's)
    assert lib.headloss_fp8_test_inject(-1, 0) == 0
    assert torch.equal(head.logits(x), want) and head.device_error() == 0
