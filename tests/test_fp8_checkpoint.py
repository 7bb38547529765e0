"""A checkpoint's 8-bit weight that training replaces: nothing that an earlier call may still read is freed or, being the
checkpoint's own, written to."""
import gc
import weakref

import pytest
import torch

import gradient_row_online_gb300 as pkg
from tests.test_decode_ops_binding import Matrix, head_on, machine  # noqa: F401


def test_what_a_call_may_still_read_stays(machine):  # noqa: F811
    h = head_on(machine, 0)
    h.held = True
    refs = [weakref.ref(t) for t in (h.q, h.scales, h.qt, h.scales_t)]
    h.set_weight(Matrix((300, 200)))
    gc.collect()
    assert all(r() is not None for r in refs)
    assert all(new is not r() for new, r in zip((h.q, h.scales, h.qt, h.scales_t), refs))
    after = h.q, h.qt
    h.set_weight(Matrix((300, 200)))
    assert (h.q, h.qt) == after


@pytest.mark.gpu
@pytest.mark.parametrize("V,D", [(300, 208), (100, 256), (1000, 100), (77, 33)])  # one row or column of blocks: scales that turn to themselves
@pytest.mark.parametrize("kind", [torch.float8_e4m3fn, torch.float8_e5m2])
def test_a_checkpoint_is_read_and_left(V, D, kind):
    g = torch.Generator().manual_seed(V)
    w = torch.randn(V, D, generator=g).cuda()
    made = pkg.Fp8Head(w, train=True)
    q = made.q[:, :D].view(torch.float8_e4m3fn).float().to(kind)
    scales = made.scales.clone()
    bits, before = q.view(torch.uint8).clone(), scales.clone()
    held = pkg.Fp8Head.from_quantized(q, scales, train=True)
    x, dl = torch.randn(9, D, generator=g).cuda(), torch.randn(9, V, generator=g).cuda()
    graph = torch.cuda.CUDAGraph()
    held.logits(x)
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        captured = held.logits(x), *held.backward(dl, x)
    for head in (made, held):
        head.set_weight(-3 * w)
    assert torch.equal(q.view(torch.uint8), bits) and torch.equal(scales, before)
    for a, b in ((held.logits(x), made.logits(x)), *zip(held.backward(dl, x), made.backward(dl, x))):
        assert torch.equal(a, b)
    del q, scales
    torch.cuda.synchronize()
    junk = [torch.full((V, n), 255, dtype=torch.uint8, device="cuda") for n in (D, -(-D // 16) * 16) for _ in range(4)]
    graph.replay()
    torch.cuda.synchronize()
    # the graph goes on with the checkpoint's codes
    again = pkg.Fp8Head.from_quantized(bits.view(kind), before, train=True)
    for a, b in zip(captured, (again.logits(x), *again.backward(dl, x))):
        assert torch.equal(a, b) and junk
