"""A StateReorder behind its close: no GPU, with stand-ins."""
import pytest
import torch

from tests.test_decode_ops_binding import Matrix, machine, reorder_on  # noqa: F401


def test_a_closed_reordering_refuses_its_calls(machine, monkeypatch):  # noqa: F811
    r, _ = reorder_on(machine, monkeypatch, [Matrix((8, 16))])
    p = Matrix((2, 4), torch.int32)
    assert r(p) is r.outs and len(machine.calls) == 1
    r.close()
    with pytest.raises(ValueError):
        r(p)
    r.close()
    assert len(machine.calls) == 1


def test_states_that_hold_nothing_are_reordered_by_no_call(machine, monkeypatch):  # noqa: F811
    r, made = reorder_on(machine, monkeypatch, [Matrix((8, 0))])
    assert r(Matrix((2, 4), torch.int32)) is r.outs and not made and not machine.calls
