"""Policy-gradient steps on one LM head with the library's calls alone around torch's matmul:

    logits   = hidden . weight^T              headloss_lmhead_logits (tensor cores)
    tokens, old log-probs                     HeadSampler, at each prompt's own settings
    loss, d loss / d logits                   HeadLoss (GRPO + entropy metric)
    d weight = d logits^T . hidden            torch.matmul
    norm and clipping over all gradients      GradClipper
    weight  -= rate * d weight

The task: every prompt (a hidden state) is rewarded for tokens of its own residue class modulo
4, several samples a prompt make a group, and a sample's advantage is its reward against its
group's mean.  Run it with `python examples/policy_step.py [steps]` on a GPU.
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import gradient_row_online_gb300 as pkg  # noqa: E402
from gradient_row_online_gb300 import headloss as hl  # noqa: E402


class Policy:
    def __init__(self, prompts=32, group=16, hidden=128, vocab=2048, rate=10.0, max_norm=0.1,
                 seed=0):
        g = torch.Generator("cuda").manual_seed(seed)
        self.g, self.group, self.rate, self.max_norm = g, group, rate, max_norm
        self.n, self.d, self.v = prompts * group, hidden, vocab
        state = torch.randn(prompts, hidden, generator=g, device="cuda")
        self.hidden = state.repeat_interleave(group, 0).bfloat16()
        self.weight = torch.randn(vocab, hidden, generator=g, device="cuda") / hidden ** 0.5
        self.scale = torch.ones(vocab, device="cuda")  # a second, small parameter: a logit scale a token
        self.want = torch.arange(prompts, device="cuda").repeat_interleave(group) % 4
        self.logits = torch.empty(self.n, vocab, dtype=torch.bfloat16, device="cuda")
        self.stats = torch.empty(self.n, vocab // 256, 2, device="cuda")
        self.err = torch.zeros(1, dtype=torch.int32, device="cuda")
        self.grad = torch.empty_like(self.logits)
        self.sampler = pkg.HeadSampler()
        self.loss = pkg.HeadLoss(
            hl.HEADLOSS_GRPO | hl.HEADLOSS_GRPO_STATS | hl.HEADLOSS_ENTROPY,
            hl.make_weights(ce=0.0, grpo=1.0, entropy=0.0))
        self.d_weight = torch.empty_like(self.weight)
        self.d_scale = torch.empty_like(self.scale)
        self.clipper = pkg.GradClipper([self.d_weight, self.d_scale])

    def step(self):
        """One step; what it saw, as device tensors."""
        head = (self.weight * self.scale[:, None]).bfloat16()
        hl.headloss_lmhead_logits(self.hidden, head, self.n, self.d, self.v, self.logits,
                                  self.stats, self.err)
        # half of each group explores at a higher temperature, none draws from the far tail
        t = torch.where(torch.arange(self.n, device="cuda") % 2 == 0, 1.0, 1.3)
        u = torch.rand(self.n, generator=self.g, device="cuda", dtype=torch.float64)
        tokens, old, _, kept = self.sampler(self.logits, u, temperature=t, top_p=0.98)
        reward = (tokens % 4 == self.want).float()
        groups = reward.view(-1, self.group)
        advantages = (groups - groups.mean(1, keepdim=True)).reshape(-1)
        scalars = self.loss(self.logits, tokens, old_logprobs=old, advantages=advantages,
                            grad_out=self.grad)
        d_head = torch.matmul(self.grad.t(), self.hidden).float()
        torch.mul(d_head, self.scale[:, None], out=self.d_weight)
        torch.sum(d_head * self.weight, 1, out=self.d_scale)
        clip = self.clipper(self.max_norm)  # in place
        self.weight -= self.rate * self.d_weight
        self.scale -= 0.01 * self.rate * self.d_scale
        return dict(reward=reward.mean(), ratio=scalars[hl.SLOTS.index("ratio_mean")],
                    entropy=scalars[hl.SLOTS.index("entropy_mean")], norm=clip[0],
                    factor=clip[1], kept=kept.float().mean())


def main(steps: int = 200) -> list:
    policy, seen = Policy(), []
    for i in range(steps):
        seen.append({k: float(v) for k, v in policy.step().items()})
        if i % 20 == 0 or i == steps - 1:
            print("step %3d  reward %.3f  entropy %.3f  ratio %.4f  kept %5.0f  norm %.4f  factor %.3f"
                  % (i, *(seen[-1][k] for k in ("reward", "entropy", "ratio", "kept", "norm", "factor"))))
    assert int(policy.err.item()) == 0 and policy.sampler.device_error() == 0
    return seen


if __name__ == "__main__":
    main(int(sys.argv[1]) if len(sys.argv) > 1 else 200)
