"""Host-side refusals of the beam search's calls: no GPU, and no address is dereferenced."""
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


def select(lib, **other):
    a = dict(logits=A, requests=2, beams=4, V=100, ld=100, dtype=1, scores=A, ended=None, eos=-1, keep=8, stay=0,
             softcap=0.0, scale=1.0, out_scores=A, parents=A, tokens=A, out_ended=None, workspace=A,
             bytes=1 << 30, stream=None)
    assert set(other) <= set(a)
    a.update(other)
    return lib.headloss_beam_select(*a.values())


@pytest.mark.parametrize("other,status", [
    (dict(requests=0), OK), (dict(requests=0, logits=None, scores=None, workspace=None), OK),
    (dict(requests=-1), ARG), (dict(requests=1 << 30), ARG), (dict(beams=0), ARG), (dict(beams=65), ARG),
    (dict(V=0), ARG), (dict(V=1 << 31, ld=1 << 31), ARG), (dict(ld=99), ARG), (dict(keep=0), ARG),
    (dict(keep=129), ARG), (dict(stay=1), ARG), (dict(stay=2, keep=4), ARG), (dict(eos=100), ARG),
    (dict(eos=-2), ARG), (dict(ended=A), ARG), (dict(softcap=-1.0), ARG), (dict(softcap=float("nan")), ARG),
    (dict(softcap=1e-39), ARG), (dict(scale=0.0), ARG), (dict(scale=float("inf")), ARG), (dict(scale=3e38), ARG),
    (dict(logits=None), ARG), (dict(scores=None), ARG), (dict(out_scores=None), ARG), (dict(parents=None), ARG),
    (dict(tokens=None), ARG), (dict(workspace=None), ARG), (dict(bytes=64), ARG), (dict(dtype=3), DTYPE),
    (dict(logits=A + 1), ALIGN), (dict(logits=A + 2, dtype=0), ALIGN), (dict(scores=A + 2), ALIGN),
    (dict(out_scores=A + 1), ALIGN), (dict(parents=A + 2), ALIGN), (dict(tokens=A + 4), ALIGN),
    (dict(workspace=A + 8), ALIGN)])
def test_select_refuses(lib, other, status):
    assert select(lib, **other) == status


def test_workspace(lib):
    need = lib.headloss_beam_workspace
    assert need(0, 4, 100, 1, 8) == 0
    assert need(2, 4, 100, 1, 8) > 0
    for bad in ((-1, 4, 100, 1, 8), (2, 0, 100, 1, 8), (2, 4, 0, 1, 8), (2, 4, 100, 3, 8), (2, 4, 100, 1, 0),
                (1 << 25, 64, 1 << 30, 1, 8)):
        assert need(*bad) == -1


def test_reorder_refuses(lib):
    out = ctypes.c_void_p()
    state = (hlb.headloss_state * 2)()
    create = lib.headloss_reorder_create
    for s in state:
        s.state, s.out, s.outer, s.positions, s.run_bytes, s.row_stride = A, A, 1, 1, 16, 16
    assert create(None, 1, 4, ctypes.byref(out)) == ARG
    assert create(state, 0, 4, ctypes.byref(out)) == ARG
    assert create(state, (1 << 20) + 1, 4, ctypes.byref(out)) == ARG
    assert create(state, 2, 0, ctypes.byref(out)) == ARG
    assert create(state, 2, 65, ctypes.byref(out)) == ARG
    assert create(state, 2, 4, None) == ARG
    for name, value in (("state", None), ("out", None), ("outer", -1), ("positions", -1), ("run_bytes", -1),
                        ("row_stride", -16), ("outer_stride", -1), ("position_stride", -1)):
        keep = getattr(state[1], name)
        setattr(state[1], name, value)
        assert create(state, 2, 4, ctypes.byref(out)) == ARG, name
        setattr(state[1], name, keep)
    assert lib.headloss_reorder(None, A, 1, None, None, None) == ARG
    lib.headloss_reorder_destroy(None)
