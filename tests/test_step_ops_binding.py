"""What HeadSampler and GradClipper check and select before they call the library: no GPU, with
stand-ins for tensors of several devices, and calls that are recorded instead of made."""
import contextlib

import pytest
import torch

from gradient_row_online_gb300 import build as B
from gradient_row_online_gb300 import headloss as hlb


class Tensor:
    """What the binding reads of a tensor."""

    def __init__(self, shape, dtype=torch.float32, device=0, contiguous=True):
        self.shape, self.dtype, self.index, self.dense = tuple(shape), dtype, device, contiguous
        self.is_cuda = device >= 0
        self.device = torch.device("cuda", device) if device >= 0 else torch.device("cpu")

    def dim(self):
        return len(self.shape)

    def numel(self):
        n = 1
        for s in self.shape:
            n *= s
        return n

    def stride(self, i):
        return 1 if i == len(self.shape) - 1 else self.shape[-1]

    def get_device(self):
        return self.index

    def is_contiguous(self):
        return self.dense

    def data_ptr(self):
        return 1 << 12


class Stream:
    def __init__(self, device):
        self.device = torch.device("cuda", device)


class Machine:
    """The current device and stream, and the calls made with them."""

    def __init__(self):
        self.device, self.stream, self.calls, self.clippers = 0, None, [], []

    @contextlib.contextmanager
    def on_device(self, index):
        before, self.device = self.device, index
        yield
        self.device = before

    @contextlib.contextmanager
    def on_stream(self, stream):
        before = self.device, self.stream
        if stream is not None:
            self.device, self.stream = stream.device.index, stream
        yield
        self.device, self.stream = before

    def call(self, name):
        def f(*args):
            self.calls.append((name, self.device, self.stream, args))
            return 0
        return f


@pytest.fixture
def machine(monkeypatch):
    B.build()
    m = Machine()
    monkeypatch.setattr(torch.cuda, "device", m.on_device)
    monkeypatch.setattr(torch.cuda, "stream", m.on_stream)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: m.device)
    monkeypatch.setattr(hlb, "_current_device", lambda: m.device, raising=False)
    monkeypatch.setattr(hlb, "_raw_stream", lambda index: ("stream", index, m.device, m.stream))

    def create(n):
        m.calls.append(("create", m.device, m.stream, (n,)))
        return 1
    monkeypatch.setattr(hlb, "headloss_clip_create", create)
    monkeypatch.setattr(hlb, "headloss_clip_destroy", lambda h: None)
    yield m
    for c in m.clippers:
        c.h = None  # no handle of the library's


def sampler_on(machine, index):
    s = object.__new__(hlb.HeadSampler)
    s.softcap, s.logits_scale = 0.0, 1.0
    s.err = Tensor((1,), torch.int32, index)
    s.device, s.index = torch.device("cuda", index), index
    s._call = machine.call("sample")
    s._empty = lambda n, dtype, device: Tensor((n,), dtype, device.index)
    s._f32, s._i32, s._f64, s._i64 = torch.float32, torch.int32, torch.float64, torch.int64
    s._codes = {torch.float32: 0, torch.bfloat16: 1, torch.float16: 2}
    return s


def clipper_on(machine, index, n=2):
    c = hlb.GradClipper([Tensor((5,), device=index) for _ in range(n)], max_grads=4)
    machine.clippers.append(c)
    c._call = machine.call("clip")
    c._empty = lambda n, dtype, device: Tensor((n,), dtype, device.index)
    return c


@pytest.mark.parametrize("current,index", [(0, 0), (0, 1), (1, 0)])
def test_the_sampler_calls_on_its_own_device(machine, current, index):
    s = sampler_on(machine, index)
    machine.device = current
    s(Tensor((3, 10), device=index), Tensor((3,), torch.float64, index))
    (name, device, _, args), = machine.calls
    assert name == "sample" and device == index and args[-1] == ("stream", index, index, None)
    assert machine.device == current


@pytest.mark.parametrize("current,index", [(0, 0), (0, 1), (1, 0)])
def test_the_clipper_creates_and_calls_on_its_gradients_device(machine, current, index):
    machine.device = current
    c = clipper_on(machine, index)
    c(1.0)
    (_, created, _, _), (_, called, _, args) = machine.calls
    assert created == called == index and args[-1] == ("stream", index, index, None)
    assert machine.device == current


def test_a_stream_of_the_operators_device_is_taken(machine):
    side = Stream(1)
    sampler_on(machine, 1)(Tensor((3, 10), device=1), Tensor((3,), torch.float64, 1), stream=side)
    clipper_on(machine, 1)(1.0, stream=side)
    for name, device, stream, args in machine.calls:
        if name != "create":
            assert device == 1 and stream is side and args[-1] == ("stream", 1, 1, side)
    assert machine.device == 0 and machine.stream is None


def test_a_stream_of_another_device_is_refused(machine):
    s, c = sampler_on(machine, 1), clipper_on(machine, 1)
    machine.calls.clear()
    with pytest.raises(ValueError):
        s(Tensor((3, 10), device=1), Tensor((3,), torch.float64, 1), stream=Stream(0))
    with pytest.raises(ValueError):
        c(1.0, stream=Stream(0))
    assert not machine.calls


def test_tensors_of_another_device_are_refused(machine):
    s = sampler_on(machine, 1)
    for x, u in ((0, 1), (1, 0), (-1, 1), (1, -1)):
        with pytest.raises(ValueError):
            s(Tensor((3, 10), device=x), Tensor((3,), torch.float64, u))
    assert not machine.calls


def test_gradients_of_two_devices_are_refused(machine):
    for devices in ((0, 1), (1, 0), (0, -1)):
        with pytest.raises(ValueError):
            hlb.GradClipper([Tensor((5,), device=d) for d in devices])
    assert not machine.calls


def test_binding_to_another_device_than_the_workspaces_is_refused(machine):
    c = clipper_on(machine, 1)
    with pytest.raises(ValueError):
        c.bind([Tensor((5,), device=0)])
    c.bind([Tensor((7,), device=1)])
    c.bind([])  # stays on its device
    c(1.0, stats=Tensor((2,), device=1))
    assert machine.calls[-1][1] == 1


@pytest.mark.parametrize("stats", [Tensor((2,), torch.float64), Tensor((2,), torch.int32), Tensor((1,)),
                                   Tensor((3,)), Tensor((0,)), Tensor((2,), device=1), Tensor((2,), device=-1),
                                   Tensor((2,), contiguous=False)])
def test_stats_that_the_call_cannot_write_are_refused(machine, stats):
    c = clipper_on(machine, 0)
    machine.calls.clear()
    with pytest.raises(ValueError):
        c(1.0, stats=stats)
    assert not machine.calls
    mine = Tensor((2,))
    assert c(1.0, stats=mine) is mine and len(machine.calls) == 1


def test_gradients_and_outputs_from_generators(machine):
    c = hlb.GradClipper((Tensor((n,)) for n in (3, 4)), (Tensor((n,)) for n in (3, 4)))
    machine.clippers.append(c)
    assert c.max_grads == 2 and [g.shape for g in c.grads] == [(3,), (4,)] and len(c.outs) == 2
