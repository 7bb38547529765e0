"""Host-side refusals of headloss_sample and headloss_clip_grads: no GPU, and
no address is dereferenced."""
import ctypes

import pytest

from gradient_row_online_gb300 import build as B
from gradient_row_online_gb300 import headloss as hlb

OK, ARG, DTYPE, ALIGN = (hlb.HEADLOSS_OK, hlb.HEADLOSS_ERR_ARG, hlb.HEADLOSS_ERR_DTYPE,
                         hlb.HEADLOSS_ERR_ALIGN)
A = 1 << 12  # an aligned address


@pytest.fixture(scope="module")
def lib():
    B.build()
    return hlb.load_library()


def sample(lib, **other):
    a = dict(logits=A, N=2, V=100, ld=100, dtype=1, uniforms=A, temperature=None, top_k=None,
             top_p=None, min_p=None, softcap=0.0, scale=1.0, tokens=A, logprobs=None, draw=None,
             kept=None, err=A, stream=None)
    assert set(other) <= set(a)
    a.update(other)
    return lib.headloss_sample(*a.values())


@pytest.mark.parametrize("other,status", [
    (dict(N=0), OK), (dict(N=0, logits=None, uniforms=None, tokens=None, err=None), OK),
    (dict(N=-1), ARG), (dict(V=0), ARG), (dict(V=1 << 31, ld=1 << 31), ARG), (dict(ld=99), ARG),
    (dict(N=1 << 31), ARG),
    (dict(softcap=-1.0), ARG), (dict(softcap=float("nan")), ARG), (dict(scale=0.0), ARG),
    (dict(scale=float("inf")), ARG), (dict(logits=None), ARG), (dict(uniforms=None), ARG),
    (dict(tokens=None), ARG), (dict(err=None), ARG), (dict(dtype=3), DTYPE), (dict(dtype=-1), DTYPE),
    (dict(logits=A + 1), ALIGN), (dict(logits=A + 2, dtype=0), ALIGN), (dict(uniforms=A + 4), ALIGN),
    (dict(tokens=A + 4), ALIGN), (dict(top_k=A + 2), ALIGN), (dict(logprobs=A + 1), ALIGN),
    (dict(kept=A + 2), ALIGN), (dict(err=A + 2), ALIGN)])
def test_sample_refuses(lib, other, status):
    assert sample(lib, **other) == status


def test_clip_refuses(lib):
    out = ctypes.c_void_p()
    assert lib.headloss_clip_create(0, ctypes.byref(out)) == ARG
    assert lib.headloss_clip_create(1 << 25, ctypes.byref(out)) == ARG
    assert lib.headloss_clip_create(4, None) == ARG
    assert lib.headloss_clip_grads(None, None, 0, 1.0, 1.0, A, None) == ARG
    lib.headloss_clip_destroy(None)
