"""Reordering of states that share memory: a cache that several layers use is moved once, what overlaps otherwise is refused."""
import pytest
import torch

import gradient_row_online_gb300 as pkg
from gradient_row_online_gb300 import headloss as hl

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("beams,R", [(4, 3), (17, 2)])
@pytest.mark.parametrize("inplace", [True, False])
def test_a_cache_of_several_layers_is_moved_once(beams, R, inplace):
    g = torch.Generator().manual_seed(beams)
    cache, other = (torch.randn(R * beams, 3, 400, 64, generator=g).bfloat16().cuda() for _ in range(2))
    before, rest = cache.clone(), other.clone()
    listed = [cache, other, cache, cache.view(cache.shape), cache]
    outs = None
    if not inplace:
        a, b = torch.zeros_like(cache), torch.zeros_like(cache)
        outs = [a, b, a, a, a]
    reorder = pkg.StateReorder(listed, beams, outs, axis=2)
    parents = torch.randint(0, beams, (R, beams), generator=g, dtype=torch.int32).cuda()  # any map: no row need keep its place
    rows = (parents.long() + beams * torch.arange(R, device="cuda")[:, None]).view(-1)
    for _ in range(3):
        got = reorder(parents)
        before, rest = (before[rows], rest[rows]) if inplace else (before, rest)
        want, want_rest = (before, rest) if inplace else (before[rows], rest[rows])
        assert torch.equal(got[0], want) and torch.equal(got[1], want_rest) and torch.equal(got[4], want)


def test_states_that_overlap_are_refused():
    t = torch.zeros(8, 6, 10, device="cuda")
    u = torch.zeros_like(t)
    p = torch.tensor([[1, 0, 3, 2]] * 2, dtype=torch.int32, device="cuda")
    t[:] = torch.arange(8.0, device="cuda")[:, None, None]
    before = t.clone()
    for states, outs in (([t, t[:, 1:]], None), ([t[:, :4], t[:, 3:]], None), ([t, u], [u, t]), ([t], [t.view(-1)[60:].new_zeros(0)]),
                         ([t, u], [u, u])):
        with pytest.raises((hl.HeadlossError, ValueError)):
            pkg.StateReorder(states, 4, outs)(p)
    assert torch.equal(t, before)
    pkg.StateReorder([t[:, :4], t[:, 4:]], 4)(p)
    assert torch.equal(t, before[[1, 0, 3, 2, 5, 4, 7, 6]])
    pkg.StateReorder([t.view(8, 60), t], 4)(p)  # rows of the same bytes, in another shape
    assert torch.equal(t, before)


def test_rows_that_the_call_does_not_reach_may_be_shared():
    buf = torch.arange(12.0, device="cuda")[:, None].repeat(1, 5)
    reorder = pkg.StateReorder([buf[:8], buf[4:]], 4)
    p = torch.tensor([[1, 0, 3, 2]], dtype=torch.int32, device="cuda")
    reorder(p)
    assert buf[:, 0].tolist() == [1, 0, 3, 2, 5, 4, 7, 6, 8, 9, 10, 11]
    with pytest.raises(hl.HeadlossError):
        reorder(p.repeat(2, 1))
    reorder(p)
    assert buf[:, 0].tolist() == [0, 1, 2, 3, 4, 5, 6, 7, 8, 9, 10, 11]
