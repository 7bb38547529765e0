"""A beam search's selection against its definition in 64 bits, and the reordering of states.

Tolerance of a score: the row's sum of exponentials is held in fp32. An exponential's argument and
value are off by 2^-22 relative, 64 of them are added a thread and 13 partial sums behind that (2^-24 each),
in all 2^-17 of the sum at most; under a cap its tanh adds 2^-21 of cap * scale. The score itself is rounded
once. Beams' candidates nearer than that may stand in either order; those of one beam may not."""
import math

import pytest
import torch

import gradient_row_online_gb300 as pkg
from gradient_row_online_gb300 import headloss as hl

pytestmark = pytest.mark.gpu


def definition(logits, scores, ended, eos, keep, cap, scale):
    """For each request the candidates in order: [(score, beam, x, token)], all of them that could be kept."""
    R, B = scores.shape
    out = []
    x64 = logits.double().cpu()
    for r in range(R):
        found = []
        for b in range(B):
            s = float(scores[r, b])
            if not s > -math.inf:
                continue
            if ended is not None and bool(ended[r, b]):
                found.append((s, b, 0.0, eos))
                continue
            x = torch.where(x64[r * B + b].isnan(), -math.inf, x64[r * B + b])
            top = x.max()
            if top == -math.inf:
                continue
            if cap:
                z = cap * torch.tanh(x / cap)
                d = torch.where(x == -math.inf, -math.inf, (z - z.max()) * scale)
            else:
                d = torch.where(x == top, 0.0, (x - top) * scale)
            lse = torch.log(torch.exp(d).sum())
            order = torch.argsort(x, descending=True, stable=True)[:keep].tolist()
            found += [(s + float(d[j] - lse), b, float(x[j]), j) for j in order if d[j] > -math.inf]
        found.sort(key=lambda c: (-c[0], c[1], -c[2], c[3]))
        out.append(found)
    return out


def check(logits, scores, ended, eos, keep, cap, scale, got, stay=False):
    R, B = scores.shape
    gs, gp, gt, ge = (t.cpu() for t in got)
    tol = 2.0 ** -17 * (1 + cap * scale / 8)
    for r, want in enumerate(definition(logits, scores, ended, eos, keep, cap, scale)):
        rows = list(zip(gs[r].tolist(), gp[r].tolist(), gt[r].tolist(), ge[r].tolist()))
        if stay:
            kept = [c for c in rows if c[1] >= 0]
            parents = {c[1] for c in kept}
            for p in parents:  # a parent that goes on has a child in its place, the best of its children
                mine = [c for c in kept if c[1] == p]
                assert rows[p][1] == p and rows[p][0] == max(c[0] for c in mine)
            rest = [i for i in range(B) if i not in parents]
            others = [rows[i] for i in rest]
            real = [c for c in others if c[1] >= 0]
            assert others[:len(real)] == real and [c[0] for c in real] == sorted((c[0] for c in real), reverse=True)
            rows = sorted(kept, key=lambda c: -c[0]) + [c for c in rows if c[1] < 0]
        n = min(keep, len(want))
        for c in rows[n:]:
            assert c == (-math.inf, -1, -1, False)
        taken = []
        for k in range(n):
            s, p, t, e = rows[k]
            exact = {(c[1], c[3]): c for c in want}
            assert (p, t) in exact, (r, k, rows[k])
            c = exact[p, t]
            assert c[0] == s or abs(s - c[0]) <= tol + abs(c[0]) * 2.0 ** -23, (r, k, s, c)
            assert e == (eos >= 0 and t == eos)
            # the one that stands here by the definition, or as near as the tolerance
            assert (p, t) == (want[k][1], want[k][3]) or abs(c[0] - want[k][0]) <= 2 * tol + abs(c[0]) * 2.0 ** -22, (r, k)
            taken.append((p, t))
        assert len(set(taken)) == n
        for b in range(B):  # within a beam the order is exact
            mine = [x for x in taken if x[0] == b]
            if not stay:
                assert mine == [(c[1], c[3]) for c in want if c[1] == b][:len(mine)]
            else:
                assert sorted(mine) == sorted([(c[1], c[3]) for c in want if c[1] == b][:len(mine)])


def make(R, B, V, dtype, seed, pad=0, shift=0, spread=3.0):
    g = torch.Generator().manual_seed(seed)
    x = (spread * torch.randn(R * B, V + pad + shift, generator=g)).to(dtype).cuda()[:, shift:shift + V]
    return x, (-5.0 * torch.rand(R, B, generator=g)).cuda(), g


@pytest.mark.parametrize("R,B,V", [(1, 1, 1), (1, 4, 7), (3, 2, 100), (2, 5, 4097), (1, 3, 32003), (2, 1, 70001)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("cap,scale,pad,shift", [(0.0, 1.0, 0, 0), (5.0, 0.7, 3, 1)])
def test_selection(R, B, V, dtype, cap, scale, pad, shift):
    x, s, _ = make(R, B, V, dtype, R + B + V, pad, shift)
    for keep in {1, B, 2 * B}:
        got = pkg.BeamSelector(B, keep, cap, scale)(x, s)
        check(x, s, None, -1, keep, cap, scale, got)
    check(x, s, None, -1, B, cap, scale, pkg.BeamSelector(B, softcap=cap, logits_scale=scale, stay=True)(x, s), stay=True)


@pytest.mark.parametrize("B,keep", [(16, 16), (16, 17), (64, 128), (33, 64), (7, 100)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_many_beams(B, keep, dtype):
    x, s, _ = make(2, B, 5000, dtype, B + keep)
    check(x, s, None, -1, keep, 0.0, 1.0, pkg.BeamSelector(B, keep)(x, s))


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("stay", [False, True])
def test_ended_dead_masked_and_forbidden(dtype, stay):
    R, B, V, eos = 6, 4, 3001, 5
    x, s, g = make(R, B, V, dtype, 11)
    ended = torch.zeros(R, B, dtype=torch.bool)
    s[0, 1:] = -math.inf                       # a first step
    s[1, :] = -math.inf                        # nothing lives
    ended[2, 1], ended[2, 3] = True, True
    ended[3, :] = True                         # all have ended
    s[3, 2] = -math.inf                        # and one of them is dead
    x[4 * B:5 * B, :] = -math.inf              # nothing is allowed
    x[4 * B + 2, 77] = 1.0                     # but one token
    x[5 * B, :] = -math.inf
    x[5 * B + 1, 2:] = math.nan
    x[5 * B + 2, ::2] = torch.finfo(dtype).min
    s[5, 3] = math.nan
    x[2 * B, eos] = 30.0                       # ends here
    ended = ended.cuda()
    x[0, 9] = math.nan
    got = pkg.BeamSelector(B, eos=eos, stay=stay)(x, s, ended)
    check(x, s, ended, eos, B, 0.0, 1.0, got, stay)


def test_infinities():
    B, V = 2, 900
    x, s, _ = make(1, B, V, torch.float32, 4)
    x[0, 17], x[0, 600] = math.inf, math.inf
    for cap in (0.0, 8.0):
        check(x, s, None, -1, 5, cap, 1.0, pkg.BeamSelector(B, 5, cap)(x, s))


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("keep", [4, 16, 40])
@pytest.mark.parametrize("kind", ["flat", "few", "narrow", "rising", "falling"])
def test_equal_logits_and_crowded_slices(dtype, keep, kind):
    R, B, V = 2, 4, 40000
    x, s, g = make(R, B, V, dtype, keep)
    if kind == "flat":
        x.fill_(0.25)
    elif kind == "few":
        x.copy_(torch.randint(0, 3, x.shape, generator=g).to(dtype))
    elif kind == "narrow":  # all that is allowed lies with a few threads
        x[:, :8] = -math.inf
        x[:, 80:] = -math.inf
    elif kind == "rising":
        x.copy_(torch.linspace(-9, 9, V).to(dtype))
    else:
        x.copy_(torch.linspace(9, -9, V).to(dtype))
    check(x, s, None, -1, keep, 0.0, 1.0, pkg.BeamSelector(B, keep)(x, s))


def test_too_many_equal_scores_to_rank():
    """Equal beams of equal logits: every candidate ties, beam and token decide."""
    x = torch.zeros(64, 70000).bfloat16().cuda()
    s = torch.zeros(1, 64).cuda()
    _, p, t, _ = pkg.BeamSelector(64, 128)(x, s)
    assert (p == 0).all() and torch.equal(t[0].cpu(), torch.arange(128))


def test_rounds_of_scores_do_not_decide_between_beams():
    """Two beams whose best candidates differ by less than fp32 shows."""
    x = torch.full((2, 1000), -30.0).cuda()
    x[0, 3], x[1, 5] = 2.0, 2.0
    x[1, 900] = -29.9999  # takes 2e-18 of the mass more than its like
    s = torch.tensor([[-1e4, -1e4]]).cuda()
    _, p, t, _ = pkg.BeamSelector(2)(x, s)
    assert p.tolist() == [[0, 1]] and t.tolist() == [[3, 5]]


def test_outputs_in_place_and_given():
    x, s, _ = make(3, 4, 5000, torch.bfloat16, 8)
    sel = pkg.BeamSelector(4, eos=1)
    ended = torch.zeros(3, 4, dtype=torch.bool, device="cuda")
    want = sel(x, s, ended)
    out = (s, torch.empty_like(want[1]), torch.empty_like(want[2]), ended)
    got = sel(x, s, ended, out=out)
    assert got is out and all(torch.equal(a, b) for a, b in zip(got, want))
    assert sel(x[:0], s[:0])[0].shape == (0, 4)


def test_selection_captured_and_on_a_stream():
    x, s, _ = make(2, 4, 9000, torch.bfloat16, 9)
    sel = pkg.BeamSelector(4, 8)
    want = sel(x, s)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = sel(x, s, stream=side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        held = sel(x, s)
    graph.replay()
    torch.cuda.synchronize()
    for a, b, c in zip(want, got, held):
        assert torch.equal(a, b) and torch.equal(a, c)


# ------------------------------------------------------------- reordering ----

def expected(states, outs, parents, beams, axis, begin, end):
    R = parents.shape[0]
    want = [o.clone() for o in outs]
    par = parents.cpu()
    for r in range(R):
        for b in range(beams):
            p = int(par[r, b])
            p = p if 0 <= p < beams else b
            for t, w in zip(states, want):
                if begin is None:
                    w[r * beams + b] = t[r * beams + p]
                else:
                    n = t.shape[axis]
                    lo, hi = max(0, int(begin[r])), min(n, int(end[r]))
                    if lo < hi:
                        w[r * beams + b].narrow(axis - 1, lo, hi - lo).copy_(t[r * beams + p].narrow(axis - 1, lo, hi - lo))
    return want


def random_state(g, shape, dtype):
    return (torch.randint(-100, 100, shape, generator=g).to(dtype) / (1 if dtype in (torch.int8, torch.uint8) else 8)).to(dtype).cuda()


@pytest.mark.parametrize("beams", [1, 2, 4, 5, 16, 17, 64])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32, torch.int8])
@pytest.mark.parametrize("inplace", [True, False])
def test_reorder(beams, dtype, inplace):
    g = torch.Generator().manual_seed(beams)
    R = 3
    rows = R * beams + 2  # two behind the last
    for axis, shapes in ((None, [(33, 77), (128,), (5,), (0,)]), (2, [(3, 50, 16), (2, 300, 64), (1, 7, 5)]),
                         (1, [(40, 3, 8), (9, 6)])):
        states = [random_state(g, (rows, *sh), dtype) for sh in shapes]
        outs = None if inplace else [random_state(g, (rows, *sh), dtype) for sh in shapes]
        parents = torch.randint(-1, beams + 1, (R, beams), generator=g, dtype=torch.int32).cuda()
        ranges = [(None, None)]
        if axis is not None:
            ranges += [(torch.tensor([0, 3, 6], dtype=torch.int32), torch.tensor([5, 3, 1000], dtype=torch.int32)),
                       (torch.tensor([-4, 5, 2], dtype=torch.int32), torch.tensor([1, 2, 3], dtype=torch.int32))]
        reorder = pkg.StateReorder(states, beams, outs, axis=axis)
        for begin, end in ranges:
            before = [t.clone() for t in states]
            want = expected(before, [o.clone() for o in reorder.outs], parents, beams, axis, begin, end)
            got = reorder(parents, begin.cuda() if begin is not None else None, end.cuda() if end is not None else None)
            assert all(torch.equal(a, b) for a, b in zip(got, want))
            if not inplace:
                assert all(torch.equal(a, b) for a, b in zip(states, before))


def test_reorder_strided_states():
    """Positions before rows, views with padding, unaligned starts."""
    g = torch.Generator().manual_seed(1)
    beams, R = 4, 2
    first = random_state(g, (30, 8, 3, 10), torch.bfloat16).transpose(0, 1)      # positions outermost
    padded = random_state(g, (8, 2, 30, 24), torch.bfloat16)[..., :20]
    odd = random_state(g, (8, 2, 30 * 6 + 1), torch.bfloat16)[..., 1:].unflatten(2, (30, 6))
    parents = torch.tensor([[3, 3, 0, 1], [1, 0, 3, 2]], dtype=torch.int32).cuda()
    begin, end = torch.tensor([2, 0], dtype=torch.int32), torch.tensor([29, 7], dtype=torch.int32)
    for state, axis in ((first, 1), (padded, 2), (odd, 2)):
        want = expected([state.clone()], [state.clone()], parents, beams, axis, begin, end)
        got = pkg.StateReorder([state], beams, axis=axis)(parents, begin.cuda(), end.cuda())
        assert torch.equal(got[0], want[0])


def test_reorder_of_many_states_and_a_long_line():
    g = torch.Generator().manual_seed(2)
    states = [random_state(g, (4, 3 + i % 5), torch.float32) for i in range(400)]
    long = random_state(g, (4, 2, 9000, 24), torch.bfloat16)
    parents = torch.tensor([[2, 0, 0, 3]], dtype=torch.int32).cuda()
    want = expected(states, states, parents, 4, None, None, None)
    assert all(torch.equal(a, b) for a, b in zip(pkg.StateReorder(states, 4)(parents), want))
    want = long[[2, 0, 0, 3]]
    assert torch.equal(pkg.StateReorder([long], 4, axis=2)(parents)[0], want)


def test_reorder_captured():
    g = torch.Generator().manual_seed(3)
    state = random_state(g, (8, 6, 40), torch.bfloat16)
    out = torch.empty_like(state)
    parents = torch.zeros(2, 4, dtype=torch.int32).cuda()
    reorder = pkg.StateReorder([state], 4, [out])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        reorder(parents)
    parents.copy_(torch.tensor([[1, 1, 2, 0], [3, 2, 1, 0]]))
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, state[[1, 1, 2, 0, 7, 6, 5, 4]])


def test_refusals():
    x, s, _ = make(2, 4, 100, torch.bfloat16, 1)
    sel = pkg.BeamSelector(4)
    for bad in (lambda: sel(x[:7], s), lambda: sel(x, s[:1]), lambda: sel(x, s.double()), lambda: sel(x.t(), s),
                lambda: sel(x, s, torch.zeros(2, 4, dtype=torch.bool, device="cuda")), lambda: sel(x.cpu(), s),
                lambda: pkg.BeamSelector(0), lambda: pkg.BeamSelector(65), lambda: pkg.BeamSelector(4, 129),
                lambda: pkg.BeamSelector(4, 8, stay=True),
                lambda: sel(x, s, out=(s, s, s, s))):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(hl.HeadlossError):
        sel(x.double(), s)
    with pytest.raises(hl.HeadlossError):
        pkg.BeamSelector(4, softcap=-1.0)(x, s)
    t = torch.zeros(8, 3, 5).cuda()
    p = torch.zeros(2, 4, dtype=torch.int32).cuda()
    re = pkg.StateReorder([t], 4, axis=1)
    i = torch.zeros(2, dtype=torch.int32).cuda()
    for bad in (lambda: re(p[:, :3]), lambda: re(p.long()), lambda: re(torch.zeros(3, 4, dtype=torch.int32).cuda()),
                lambda: re(p, i), lambda: re(p, i, i[:1]), lambda: pkg.StateReorder([t], 4)(p, i, i),
                lambda: pkg.StateReorder([], 4), lambda: pkg.StateReorder([t], 4, [t.half()]),
                lambda: pkg.StateReorder([t], 4, axis=0), lambda: pkg.StateReorder([t], 4, axis=3),
                lambda: pkg.StateReorder([t.transpose(1, 2)], 4), lambda: pkg.StateReorder([t[:1].expand(8, 3, 5)], 4),
                lambda: pkg.StateReorder([t.cpu()], 4)):
        with pytest.raises(ValueError):
            bad()
