"""Beam search steps on an 8-bit head: logits, the selection, and the beams' caches reordered in place.

A stand-in for a decoder keeps a running state and a key-value cache a beam; what matters is what stands
behind the head: `Fp8Head.logits` -> `BeamSelector` -> `StateReorder`.
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import gradient_row_online_gb300 as pkg  # noqa: E402


class Decoder:
    """A toy decoder: a state of `width` a row, and a cache of (rows, heads, positions, width / heads)."""

    def __init__(self, requests, beams, width, heads, prompt, steps, vocab, eos, device="cuda", seed=0):
        g = torch.Generator(device).manual_seed(seed)
        rows = requests * beams
        self.requests, self.beams, self.position = requests, beams, prompt
        self.embedding = torch.randn(vocab, width, generator=g, device=device).to(torch.bfloat16)
        self.mix = (torch.randn(width, width, generator=g, device=device) * width ** -0.5).to(torch.bfloat16)
        start = torch.randn(requests, width, generator=g, device=device).to(torch.bfloat16)
        self.state = start.repeat_interleave(beams, 0)
        self.cache = torch.zeros(rows, heads, prompt + steps, width // heads, dtype=torch.bfloat16, device=device)
        # the beams share their prompt: only what follows it moves
        self.begin = torch.full((requests,), prompt, dtype=torch.int32, device=device)
        self.head = pkg.Fp8Head(torch.randn(vocab, width, generator=g, device=device) * width ** -0.5)
        self.selector = pkg.BeamSelector(beams, eos=eos, stay=True, device=device)
        self.reorder_state = pkg.StateReorder([self.state], beams)
        self.reorder_cache = pkg.StateReorder([self.cache], beams, axis=2)
        self.scores = torch.full((requests, beams), -torch.inf, device=device)
        self.scores[:, 0] = 0.0  # before the first step the beams are the same
        self.ended = torch.zeros(requests, beams, dtype=torch.bool, device=device)

    def step(self):
        """One token a beam; returns (parents, tokens)."""
        logits = self.head.logits(self.state)
        self.scores, parents, tokens, self.ended = self.selector(logits, self.scores, self.ended)
        end = torch.full_like(self.begin, self.position)
        self.reorder_state(parents)
        self.reorder_cache(parents, self.begin, end)
        row = self.embedding[tokens.view(-1).clamp(min=0)]
        new = torch.tanh(self.state @ self.mix + row)
        self.cache[:, :, self.position] = new.view(self.cache.shape[0], self.cache.shape[1], -1)
        self.state.copy_(new)
        self.position += 1
        return parents, tokens


def main(requests=4, beams=4, steps=16):
    decoder = Decoder(requests, beams, 1024, 8, 64, steps, 32000, eos=2)
    sequences = None
    for _ in range(steps):
        parents, tokens = decoder.step()
        if sequences is None:
            sequences = tokens[..., None]
        else:
            kept = torch.take_along_dim(sequences, parents.long()[..., None].clamp(min=0), 1)
            sequences = torch.cat((kept, tokens[..., None]), 2)
    assert decoder.head.device_error() == 0
    best = decoder.scores.argmax(1)
    for r in range(requests):
        print("request %d: %.3f %s" % (r, float(decoder.scores[r, best[r]]), sequences[r, best[r]].tolist()))


if __name__ == "__main__":
    main()
