"""A beam search's selection among zeros of both signs, which are equal: beam and token decide."""
import math

import pytest
import torch

import gradient_row_online_gb300 as pkg

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("keep", [1, 8, 40])
@pytest.mark.parametrize("cap", [0.0, 30.0])
@pytest.mark.parametrize("V", [50, 20000])
def test_logits_of_both_zeros(dtype, keep, cap, V):
    g = torch.Generator().manual_seed(V + keep)
    x = torch.where(torch.rand(4, V, generator=g) < 0.5, -0.0, 0.0)
    x[2] = torch.where(torch.rand(V, generator=g) < 0.5, -1.0, x[2])  # zeros, and half of what there is
    x[3] = -math.inf
    x[3, V // 3::3] = x[0, V // 3::3]
    want = x.argsort(dim=1, descending=True, stable=True)[:, :keep]
    score, parent, token, _ = pkg.BeamSelector(1, keep, cap)(x.to(dtype).cuda(), torch.zeros(4, 1, device="cuda"))
    real = torch.arange(keep) < (x > -math.inf).sum(1, keepdim=True)
    assert torch.equal(token.cpu(), torch.where(real, want, -1))
    assert torch.equal(parent.cpu(), torch.where(real, 0, -1).int())


def test_scores_of_both_zeros():
    """A log-prob of 0 behind scores of either sign: beams that have ended, and rows of one token."""
    scores = torch.tensor([[-0.0, 0.0, -0.0, 0.0]]).cuda()
    x = torch.full((4, 300), -math.inf)
    x[:, 7] = 1.0
    _, p, t, _ = pkg.BeamSelector(4, eos=7)(x.cuda(), scores)
    assert p.tolist() == [[0, 1, 2, 3]] and t.tolist() == [[7] * 4]
    ended = torch.tensor([[True, True, False, True]]).cuda()
    _, p, t, _ = pkg.BeamSelector(4, 3, eos=7)(x.cuda(), scores, ended)
    assert p.tolist() == [[0, 1, 2]] and t.tolist() == [[7] * 3]
