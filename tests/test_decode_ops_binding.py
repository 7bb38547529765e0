"""What Fp8Head, BeamSelector and StateReorder check and select before they call the library: no GPU, with
stand-ins for tensors of several devices, and calls that are recorded instead of made."""
import pytest
import torch

from gradient_row_online_gb300 import headloss as hlb
from tests.test_step_ops_binding import Machine, Stream, Tensor, machine  # noqa: F401


class Matrix(Tensor):
    """A stand-in with a strides tuple, as the binding reads it."""

    def __init__(self, shape, dtype=torch.float32, device=0, contiguous=True, strides=None):
        super().__init__(shape, dtype, device, contiguous)
        if strides is None:
            strides, n = [], 1
            for s in reversed(self.shape):
                strides.insert(0, n)
                n *= max(s, 1)
        self.strides = tuple(strides)

    def stride(self, i=None):
        return self.strides if i is None else self.strides[i]

    def element_size(self):
        return torch.empty(0, dtype=self.dtype).element_size()

    def zero_(self):
        return self


def empty(*shape, dtype, device):
    shape = shape[0] if len(shape) == 1 and not isinstance(shape[0], int) else shape
    return Matrix(shape, dtype, device.index)


class Library:
    def __init__(self, m):
        self.m = m
        self.headloss_fp8_workspace = self.headloss_fp8_linear_workspace = lambda *a: 64

    def __getattr__(self, name):
        return self.m.call(name)


def head_on(m, index, train=True):
    h = object.__new__(hlb.Fp8Head)
    h.V, h.D, h.train, h.type, h.grads, h.held = 300, 200, train, hlb.HEADLOSS_E4M3, hlb.HEADLOSS_E5M2, False
    h.index, h.device = index, torch.device("cuda", index)
    h.weight_dtype = torch.bfloat16
    h._lib, h._needs, h._empty, h._u8, h._f32 = Library(m), {}, empty, torch.uint8, torch.float32
    h._codes = {torch.float32: 0, torch.bfloat16: 1, torch.float16: 2}
    h.err = Matrix((1,), torch.int32, index)
    h._make()
    return h


def selector_on(m, index, beams=4, keep=8, **more):
    s = hlb.BeamSelector(beams, keep, device=f"cuda:{index}", **more)
    s._call, s._empty = m.call("select"), empty
    return s


def reorder_on(m, monkeypatch, states, beams=4, **more):
    made = []
    monkeypatch.setattr(hlb, "headloss_reorder_create",
                        lambda table, n, b: made.append((m.device, n, b, [table[i] for i in range(n)])) or 1)
    monkeypatch.setattr(hlb, "headloss_reorder_destroy", lambda h: None)
    r = hlb.StateReorder(states, beams, **more)
    r._call = m.call("reorder")
    m.clippers.append(r)  # whose handle, none of the library's, goes before it does
    return r, made


@pytest.mark.parametrize("current,index", [(0, 0), (0, 1), (1, 0)])
def test_calls_are_made_on_the_operators_device(machine, monkeypatch, current, index):  # noqa: F811
    machine.device = current
    h = head_on(machine, index)
    x, g = Matrix((5, 200), torch.bfloat16, index), Matrix((5, 300), torch.bfloat16, index)
    h.logits(x)
    h.backward(g, x)
    h.set_weight(Matrix((300, 200), device=index))
    selector_on(machine, index)(Matrix((8, 100), device=index), Matrix((2, 4), device=index))
    r, made = reorder_on(machine, monkeypatch, [Matrix((8, 16), device=index)])
    r(Matrix((2, 4), torch.int32, index))
    assert made[0][0] == index and len(machine.calls) >= 7
    for name, device, _, args in machine.calls:
        assert device == index and args[-1] == ("stream", index, index, None), name
    assert machine.device == current


def test_a_stream_of_another_device_is_refused(machine, monkeypatch):  # noqa: F811
    h, s = head_on(machine, 1), selector_on(machine, 1)
    r, _ = reorder_on(machine, monkeypatch, [Matrix((8, 16), device=1)])
    x = Matrix((5, 200), device=1)
    for call in (lambda: h.logits(x, stream=Stream(0)), lambda: h.backward(Matrix((5, 300), device=1), x, stream=Stream(0)),
                 lambda: h.set_weight(Matrix((300, 200), device=1), stream=Stream(0)),
                 lambda: s(Matrix((8, 100), device=1), Matrix((2, 4), device=1), stream=Stream(0)),
                 lambda: r(Matrix((2, 4), torch.int32, 1), stream=Stream(0))):
        with pytest.raises(ValueError):
            call()
    assert not machine.calls
    side = Stream(1)
    h.logits(x, stream=side)
    assert machine.calls[-1][2] is side and machine.calls[-1][3][-1] == ("stream", 1, 1, side)


@pytest.mark.parametrize("x", [
    Matrix((5, 199)), Matrix((5, 200), torch.float64), Matrix((5, 200), device=1), Matrix((5, 200), device=-1),
    Matrix((200,)), Matrix((5, 200), strides=(1, 5)), Matrix((5, 200), strides=(0, 1)), Matrix((5, 200), strides=(100, 1))])
def test_hidden_states_that_the_head_cannot_take(machine, x):  # noqa: F811
    h = head_on(machine, 0)
    with pytest.raises(ValueError):
        h.logits(x)
    with pytest.raises(ValueError):
        h.backward(Matrix((5, 300)), x)
    assert not machine.calls


def test_outputs_that_the_head_cannot_write(machine):  # noqa: F811
    h = head_on(machine, 0)
    x, g = Matrix((5, 200), torch.bfloat16), Matrix((5, 300), torch.bfloat16)
    for out in (Matrix((5, 299)), Matrix((4, 300)), Matrix((5, 300), device=1), Matrix((5, 300), strides=(0, 1)),
                Matrix((5, 300), torch.int8)):
        with pytest.raises(ValueError):
            h.logits(x, out=out)
    with pytest.raises(ValueError):
        h.logits(x, out=Matrix((5, 300)), dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        h.backward(g, x, grad_weight=Matrix((200, 300)))
    with pytest.raises(ValueError):
        h.backward(g, x, grad_hidden=Matrix((5, 300)))
    with pytest.raises(ValueError):
        h.backward(Matrix((4, 300)), x)
    with pytest.raises(ValueError):
        head_on(machine, 0, train=False).backward(g, x)
    with pytest.raises(ValueError):
        h.set_weight(Matrix((300, 201)))
    assert not machine.calls
    assert h.logits(x, out=Matrix((5, 300))).dtype is torch.float32
    gh, gw = h.backward(g, x)
    assert gh.dtype is torch.bfloat16 and gw.dtype is torch.bfloat16
    h.set_weight(Matrix((300, 200)))
    assert h.backward(g, x)[1].dtype is torch.float32  # the weight's type


def test_a_checkpoints_codes_are_not_written_to(machine):  # noqa: F811
    h = head_on(machine, 0)
    h.held, before = True, h.q
    h.set_weight(Matrix((300, 200)))
    assert h.q is not before and not h.held
    after = h.q
    h.set_weight(Matrix((300, 200)))
    assert h.q is after


def test_layouts_of_states(machine, monkeypatch):  # noqa: F811
    half = torch.bfloat16
    _, made = reorder_on(machine, monkeypatch, [
        Matrix((8, 2, 50, 16), half), Matrix((8, 3, 4, 50, 16), half, strides=(9600, 3200, 800, 16, 1))], axis=2)
    with pytest.raises(ValueError):  # heads and groups that do not go as one
        reorder_on(machine, monkeypatch, [Matrix((8, 3, 4, 50, 16), half, strides=(99999, 5000, 800, 16, 1))], axis=3)
    e = made[0][3][0]
    assert (e.outer, e.positions, e.run_bytes, e.row_stride, e.outer_stride, e.position_stride) == (2, 50, 32, 3200, 1600, 32)
    _, made = reorder_on(machine, monkeypatch, [Matrix((8, 3, 4, 50, 16), half)], axis=3)
    e = made[0][3][0]
    assert (e.outer, e.positions, e.run_bytes, e.outer_stride, e.position_stride) == (12, 50, 32, 1600, 32)
    _, made = reorder_on(machine, monkeypatch, [Matrix((8, 30, 3, 10), half, strides=(30, 240, 10, 1))], axis=1)
    e = made[0][3][0]
    assert (e.outer, e.positions, e.run_bytes, e.row_stride, e.position_stride) == (1, 30, 60, 60, 480)
    _, made = reorder_on(machine, monkeypatch, [Matrix((8, 0), half), Matrix((9, 7), torch.int8)])
    (_, n, beams, table), = made
    assert n == 1 and beams == 4 and table[0].run_bytes == 7  # what holds nothing is left out


def test_calls_that_the_selection_and_the_reordering_refuse(machine, monkeypatch):  # noqa: F811
    s = selector_on(machine, 0, eos=3)
    x, before = Matrix((8, 100)), Matrix((2, 4))
    for call in (lambda: s(Matrix((7, 100)), before), lambda: s(x, Matrix((2, 3))), lambda: s(x, Matrix((2, 4), torch.float64)),
                 lambda: s(x, Matrix((2, 4), device=1)), lambda: s(x, Matrix((2, 4), contiguous=False)),
                 lambda: s(Matrix((8, 100), device=1), before), lambda: s(Matrix((8, 100), strides=(1, 8)), before),
                 lambda: s(x, before, Matrix((2, 4), torch.uint8)), lambda: s(Matrix((8, 0)), before),
                 lambda: selector_on(machine, 0)(x, before, Matrix((2, 4), torch.bool)),
                 lambda: hlb.BeamSelector(3, 4, stay=True, device="cuda:0")):
        with pytest.raises(ValueError):
            call()
    r, _ = reorder_on(machine, monkeypatch, [Matrix((9, 2, 50, 16)), Matrix((11, 5, 7, 3))], axis=2)
    p, i = Matrix((2, 4), torch.int32), Matrix((2,), torch.int32)
    for call in (lambda: r(Matrix((3, 4), torch.int32)), lambda: r(Matrix((2, 3), torch.int32)), lambda: r(Matrix((2, 4), torch.int64)),
                 lambda: r(Matrix((2, 4), torch.int32, 1)), lambda: r(p, i), lambda: r(p, i, Matrix((3,), torch.int32)),
                 lambda: r(p, i, Matrix((2,), torch.int64))):
        with pytest.raises(ValueError):
            call()
    assert not machine.calls
    assert r(p, i, i) is r.outs and len(machine.calls) == 1
