"""Host-side refusals of the 8-bit products: no GPU, and no address is dereferenced."""
import pytest
import torch

from gradient_row_online_gb300 import build as B
from gradient_row_online_gb300 import headloss as hlb

OK, ARG, DTYPE, ALIGN = (hlb.HEADLOSS_OK, hlb.HEADLOSS_ERR_ARG, hlb.HEADLOSS_ERR_DTYPE,
                         hlb.HEADLOSS_ERR_ALIGN)
A = 1 << 12  # an aligned address


@pytest.fixture(scope="module")
def lib():
    B.build()
    return hlb.load_library()


def quantize(lib, **other):
    a = dict(x=A, rows=3, cols=100, ld=100, dtype=1, type=0, q=A, ldq=112, scales=A, block=1, qt=A, ldqt=16,
             scales_t=A, block_t=128, stream=None)
    assert set(other) <= set(a)
    a.update(other)
    return lib.headloss_fp8_quantize(*a.values())


@pytest.mark.parametrize("other,status", [
    (dict(rows=0), OK), (dict(cols=0, x=None), OK), (dict(rows=-1), ARG), (dict(cols=-1), ARG),
    (dict(rows=1 << 31, ldqt=1 << 31), ARG), (dict(cols=1 << 31, ld=1 << 31, ldq=1 << 31), ARG),
    (dict(rows=1 << 30, cols=1 << 30, ld=1 << 30, ldq=1 << 30, ldqt=1 << 30), ARG), (dict(ld=99), ARG),
    (dict(x=None), ARG), (dict(q=None, qt=None), ARG), (dict(scales=None), ARG), (dict(scales_t=None), ARG),
    (dict(ldq=96), ARG), (dict(ldq=104), ALIGN), (dict(ldqt=0), ARG), (dict(ldqt=8), ALIGN),
    (dict(block=2), ARG), (dict(block_t=0), ARG), (dict(type=2), ARG), (dict(type=-1), ARG),
    (dict(dtype=3), DTYPE), (dict(x=A + 1), ALIGN), (dict(x=A + 2, dtype=0), ALIGN), (dict(q=A + 8), ALIGN),
    (dict(qt=A + 8), ALIGN), (dict(scales=A + 2), ALIGN), (dict(scales_t=A + 1), ALIGN)])
def test_quantize_refuses(lib, other, status):
    assert quantize(lib, **other) == status


def matmul(lib, **other):
    a = dict(a=A, lda=112, a_scales=A, a_type=0, b=A, ldb=112, b_scales=A, b_type=0, M=3, N=200, K=100, out=A,
             ldo=200, out_dtype=1, workspace=None, bytes=0, err=A, stream=None)
    assert set(other) <= set(a)
    a.update(other)
    return lib.headloss_fp8_matmul(*a.values())


@pytest.mark.parametrize("other,status", [
    (dict(M=0), OK), (dict(N=0, a=None, out=None, err=None), OK), (dict(M=-1), ARG), (dict(N=-1), ARG),
    (dict(K=0), ARG), (dict(K=1 << 31, lda=1 << 31, ldb=1 << 31), ARG), (dict(M=1 << 31), ARG),
    (dict(M=1 << 30, N=1 << 30, ldo=1 << 30), ARG), (dict(lda=96), ARG), (dict(ldb=96), ARG), (dict(ldo=199), ARG),
    (dict(a=None), ARG), (dict(b=None), ARG), (dict(a_scales=None), ARG), (dict(b_scales=None), ARG),
    (dict(out=None), ARG), (dict(err=None), ARG), (dict(a_type=2), ARG), (dict(b_type=-1), ARG),
    (dict(out_dtype=3), DTYPE), (dict(out_dtype=-1), DTYPE), (dict(lda=104), ALIGN), (dict(ldb=120), ALIGN),
    (dict(a=A + 8), ALIGN), (dict(b=A + 4), ALIGN), (dict(a_scales=A + 2), ALIGN), (dict(b_scales=A + 1), ALIGN),
    (dict(out=A + 1), ALIGN), (dict(out=A + 2, out_dtype=0), ALIGN), (dict(err=A + 2), ALIGN),
    (dict(workspace=A + 4), ALIGN)])
def test_matmul_refuses(lib, other, status):
    assert matmul(lib, **other) == status


def linear(lib, **other):
    a = dict(x=A, ldx=100, dtype=1, b=A, ldb=112, b_scales=A, b_type=0, M=3, N=200, K=100, out=A, ldo=200,
             out_dtype=1, workspace=A, bytes=1 << 20, err=A, stream=None)
    assert set(other) <= set(a)
    a.update(other)
    return lib.headloss_fp8_linear(*a.values())


@pytest.mark.parametrize("other,status", [
    (dict(M=0), OK), (dict(N=0, x=None, b=None, workspace=None), OK), (dict(M=-1), ARG), (dict(K=0), ARG),
    (dict(K=1 << 31, ldx=1 << 31, ldb=1 << 31), ARG), (dict(ldb=96), ARG), (dict(ldo=199), ARG), (dict(b=None), ARG),
    (dict(b_scales=None), ARG), (dict(out=None), ARG), (dict(err=None), ARG), (dict(workspace=None), ARG),
    (dict(bytes=64), ARG), (dict(b_type=3), ARG), (dict(out_dtype=3), DTYPE), (dict(ldb=104), ALIGN),
    (dict(workspace=A + 8), ALIGN), (dict(out=A + 1), ALIGN)])
def test_linear_refuses(lib, other, status):
    assert linear(lib, **other) == status


def test_workspace_refuses(lib):
    assert lib.headloss_fp8_linear_workspace(1, 1, 0) == -1
    assert lib.headloss_fp8_workspace(-1, 1, 1) == -1
    assert lib.headloss_fp8_workspace(1, 1, 0) == -1


def test_head_refuses_what_is_not_on_a_gpu():
    w = torch.zeros(8, 8)
    with pytest.raises(ValueError):
        hlb.Fp8Head(w)
    with pytest.raises(ValueError):
        hlb.Fp8Head.from_quantized(w.to(torch.float8_e4m3fn), torch.ones(1, 1))
