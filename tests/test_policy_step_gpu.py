"""The policy-step example: sampling, the loss and clipping together."""
import importlib.util
import os

import pytest

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_the_example_learns():
    spec = importlib.util.spec_from_file_location(
        "policy_step", os.path.join(ROOT, "examples", "policy_step.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    seen = m.main(120)
    # the sampler's log-probs are the loss's own: every ratio is 1 on the step they were drawn
    # for (both read the same bf16 logits; exp of a difference of two fp32 log-probs below 10)
    assert all(abs(s["ratio"] - 1.0) < 1e-4 for s in seen)
    assert all(s["factor"] <= 1.0 and s["norm"] * s["factor"] <= 0.1 * (1 + 1e-4) for s in seen)
    # chance is 1 in 4
    assert sum(s["reward"] for s in seen[-10:]) / 10 > sum(s["reward"] for s in seen[:10]) / 10 + 0.2
