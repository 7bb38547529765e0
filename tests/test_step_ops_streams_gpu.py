"""Sampling and clipping on a stream that is given: what the call makes itself (numbers as
settings, outputs) belongs to that stream, whatever the current one still has to do."""
import pytest
import torch

import gradient_row_online_gb300 as pkg
from tests.test_sample_gpu import noise

pytestmark = pytest.mark.gpu

BUSY = 400_000_000  # clock cycles, about 0.2 s
WAYS = ["stream", "handle"]


def given(side, way):
    return side if way == "stream" else side.cuda_stream


def spent(n, value, dtype, many=8):
    """Blocks of the current stream's pool that hold `value`, given back."""
    blocks = [torch.full((n,), value, dtype=dtype, device="cuda") for _ in range(many)]
    torch.cuda.synchronize()
    del blocks


@pytest.mark.parametrize("way", WAYS)
def test_a_number_is_filled_in_before_the_kernel_reads_it(way):
    x, u = noise(64, 5000, "bf16", seed=3)
    sampler = pkg.HeadSampler()
    want = [o.clone() for o in sampler(x, u, temperature=0.7, top_p=0.9)]
    side = torch.cuda.Stream()
    spent(64, 5.0, torch.float32)
    torch.cuda._sleep(BUSY)  # the current stream's fills would come after this
    got = sampler(x, u, temperature=0.7, top_p=0.9, stream=given(side, way))
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    assert sampler.device_error() == 0


@pytest.mark.parametrize("way", WAYS)
def test_a_number_stays_until_the_kernel_has_read_it(way):
    x, u = noise(64, 5000, "bf16", seed=4)
    sampler = pkg.HeadSampler()
    want = [o.clone() for o in sampler(x, u, temperature=0.7, top_p=0.9)]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        torch.cuda._sleep(BUSY)
    got = sampler(x, u, temperature=0.7, top_p=0.9, stream=given(side, way))
    later = [torch.full((64,), 5.0, device="cuda") for _ in range(64)]  # noqa: F841
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, got))


@pytest.mark.parametrize("way", WAYS)
def test_outputs_are_not_memory_that_the_current_stream_still_writes(way):
    x, u = noise(1000, 500, "bf16", seed=5)
    g = [torch.randn(70_001, device="cuda")]
    o = [torch.empty_like(g[0])]
    sampler, clipper = pkg.HeadSampler(), pkg.GradClipper(g, o)
    want = [a.clone() for a in sampler(x, u)] + [clipper(0.5).clone()]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    blocks = [torch.empty(n, dtype=d, device="cuda") for _ in range(16)
              for n, d in ((1000, torch.int64), (1000, torch.float32), (2, torch.float32))]
    torch.cuda._sleep(BUSY)
    for b in blocks:
        b.fill_(-7)
    del blocks, b
    got = [*sampler(x, u, stream=given(side, way)), clipper(0.5, stream=given(side, way))]
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, got))


@pytest.mark.parametrize("handle", [0, 1])
def test_the_default_stream_by_its_handle(handle):
    """The calls come after the default stream's work, whatever stream is current."""
    x, u = noise(64, 5000, "bf16", seed=6)
    sampler, clipper = pkg.HeadSampler(), pkg.GradClipper([x])
    want = [a.clone() for a in sampler(x, u)] + [clipper(1e9).clone()]
    late = torch.zeros_like(x)
    clipper.bind([late])
    torch.cuda.synchronize()
    torch.cuda._sleep(BUSY)
    late.copy_(x)
    with torch.cuda.stream(torch.cuda.Stream()):
        got = [*sampler(late, u, stream=handle), clipper(1e9, stream=handle)]
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, got))


@pytest.mark.parametrize("handle", [0, 1])
def test_device_error_waits_for_the_default_stream(handle):
    x, u = noise(8, 500, "bf16", seed=7)
    sampler = pkg.HeadSampler()
    bad = torch.full((8,), -1.0, device="cuda")
    torch.cuda._sleep(BUSY)
    sampler(x, u, temperature=bad)
    assert sampler.device_error(handle) == 1
    assert sampler.device_error(handle) == 0
