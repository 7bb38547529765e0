"""A beam search's selection over rows with infinite logits (an overflow in 16 bits): a row has its mass on its
infinities, and where those are fewer than what is kept the rest is -inf, -1, -1, in order or with `stay`."""
import math

import pytest
import torch

import gradient_row_online_gb300 as pkg

pytestmark = pytest.mark.gpu


def rows(live, beams, V, dtype, each, seed):
    """Scores and logits of one request: `live` beams with `each` infinities, all others dead."""
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(beams, V, generator=g)
    at = [sorted(torch.randperm(V, generator=g)[:each].tolist()) for _ in range(beams)]
    for row, places in zip(x, at):
        row[places] = math.inf
    scores = torch.full((1, beams), -math.inf)
    order = torch.randperm(beams, generator=g)[:live].tolist()
    scores[0, order] = -torch.rand(live, generator=g)
    want = sorted((-(float(scores[0, b]) - math.log(each)), b, t) for b in order for t in at[b])
    return x.to(dtype).cuda(), scores.cuda(), want


# lists of candidates that are held at once (two and one a beam), more than are ranked at once; and few
@pytest.mark.parametrize("live,beams,keep,V", [(16, 16, 32, 32000), (20, 32, 64, 9000), (9, 64, 128, 9000),
                                               (64, 64, 128, 32000), (3, 4, 8, 9000)])
@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16, torch.float32])
@pytest.mark.parametrize("each", [1, 2])
def test_fewer_infinities_than_kept(live, beams, keep, V, dtype, each):
    x, scores, want = rows(live, beams, V, dtype, each, live + keep)
    s, p, t, e = (a[0].cpu() for a in pkg.BeamSelector(beams, keep)(x, scores))
    n = min(keep, len(want))
    assert p[:n].tolist() == [w[1] for w in want[:n]] and t[:n].tolist() == [w[2] for w in want[:n]]
    # a sum of one or two equal terms and its logarithm: a rounding each, beside the score's own
    assert all(abs(float(a) + w[0]) <= 2.0 ** -22 * (1 + abs(w[0])) for a, w in zip(s, want))
    assert (s[n:] == -math.inf).all() and (p[n:] == -1).all() and (t[n:] == -1).all() and not e.any()


@pytest.mark.parametrize("live,beams,V", [(20, 32, 32000), (9, 64, 9000), (1, 64, 9000), (40, 64, 70001)])
@pytest.mark.parametrize("dtype", [torch.float16, torch.float32])
def test_places_that_nothing_takes(live, beams, V, dtype):
    """Two requests in one call, so that what does not belong to the first one's places would be seen in the second's."""
    x, scores, want = rows(live, beams, V, dtype, 1, live)
    x, scores = x.repeat(2, 1), scores.repeat(2, 1)
    guard = 64
    bufs = [torch.full((2 * beams + 2 * guard,), 77, dtype=d, device="cuda")
            for d in (torch.float32, torch.int32, torch.int64)] + [torch.zeros(2 * beams + 2 * guard, dtype=torch.bool, device="cuda")]
    out = tuple(b[guard:guard + 2 * beams].view(2, beams) for b in bufs)
    s, p, t, _ = pkg.BeamSelector(beams, stay=True)(x, scores, out=out)
    token = {b: at for _, b, at in want}
    for r in range(2):
        for b in range(beams):
            if b in token:
                assert (int(p[r, b]), int(t[r, b])) == (b, token[b]) and float(s[r, b]) == float(scores[r, b])
            else:
                assert (float(s[r, b]), int(p[r, b]), int(t[r, b])) == (-math.inf, -1, -1)
    for b in bufs[:3]:
        assert (b[:guard] == 77).all() and (b[guard + 2 * beams:] == 77).all()
