"""RankStep's use of Muon's settings: they are read at every step, and what is no setting is refused when the step is built
(stand-ins for the table: no call reaches the device)."""
import pytest
import torch

from zero_partitioned_mixed_partition_amd import step


class _Table:
    made = 0

    def __init__(self, *lists):
        type(self).made += 1

    def prepare_step(self, **settings):
        return lambda: _Table.log.append(settings)


@pytest.fixture
def rank_step(monkeypatch):
    """A step of two matrices, whose Muon calls are logged, on streams 64 (the current one) and others."""
    import zero_partitioned_mixed_partition_amd as zm

    class _Stream:
        cuda_stream = 64

    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: _Stream())
    monkeypatch.setattr(step.zb, "MuonTable", _Table)
    monkeypatch.setattr(step.RankStep, "_mt_table", lambda self: type("T", (), {
        "prepare_step": lambda self, **kw: (lambda t: None)})())
    _Table.log, _Table.made = [], 0

    def build(**muon):
        plan = zm.zero_partition_plan([12, 5, 20], 1, 1)
        return step.RankStep(plan, 0, 1, step.Hyper(), 0.0, torch.device("cpu"), per_param=True,
                             muon=step.MuonHyper(**muon), muon_shapes={0: (3, 4), 2: (4, 5)})

    return build


def test_settings_assigned_between_steps_are_taken(rank_step):
    rs = rank_step(lr=1e-3)
    for change in (dict(), dict(lr=5e-4), dict(weight_decay=0.0), dict(momentum=0.9), dict(nesterov=False), dict(eps=1e-6),
                   dict(coefficients=[[2.0, -1.5, 0.5]])):
        for k, v in change.items():
            setattr(rs.muon, k, v)
        rs.adamw()
        got = _Table.log[-1]
        assert (got["lr"], got["weight_decay"], got["momentum"], got["nesterov"], got["eps"]) == (
            rs.muon.lr, rs.muon.weight_decay, rs.muon.momentum, rs.muon.nesterov, rs.muon.eps), change
        assert got["coefficients"] == tuple(tuple(s) for s in rs.muon.coefficients)
    rs.muon.coefficients[0][0] = 1.5                     # in place
    rs.adamw()
    assert _Table.log[-1]["coefficients"] == ((1.5, -1.5, 0.5),)
    assert _Table.made == 1


def test_a_step_on_another_stream_or_with_another_rate_keeps_the_table(rank_step):
    """A captured step reads the table at each replay."""
    rs = rank_step(lr=1e-3)
    rs.adamw()
    rs.adamw(stream=4096)
    rs.muon.lr = 1e-4
    rs.adamw()
    assert _Table.made == 1 and [x["lr"] for x in _Table.log] == [1e-3, 1e-3, 1e-4]


@pytest.mark.parametrize("lr", [[1e-3, 5e-4], (1e-3,), torch.ones(3), None])
def test_a_sequence_of_rates_is_refused_when_the_step_is_built(rank_step, lr):
    with pytest.raises(ValueError, match="lr is one number"):
        rank_step(lr=lr)
    rs = rank_step(lr=1e-3)
    rs.muon.lr = lr
    with pytest.raises(ValueError, match="lr is one number"):
        rs.adamw()
    assert _Table.log == [] and rs.t == 0
