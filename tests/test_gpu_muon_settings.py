"""RankStep with Muon whose settings change between steps, and a captured step beside eager ones on another stream."""
import pytest
import torch

from tests.gpu_util import needs_gpu, to_dev_u16
from tests.test_gpu_muon_step import MATRICES, build, replicas

pytestmark = [pytest.mark.gpu, needs_gpu]


@pytest.fixture(scope="module")
def zm():
    import zero_partitioned_mixed_partition_amd as m
    return m


@pytest.fixture(scope="module")
def st():
    from zero_partitioned_mixed_partition_amd import step as s
    return s


def arrays(rs):
    return rs.master_tensors + rs.exp_avg_tensors + rs.tensors


@pytest.mark.parametrize("device_step", [False, True])
def test_a_rate_assigned_between_steps(zm, st, device_step):
    """At rate 0 without decay the matrices stay where they are and the other tensors move; with the rate back both do."""
    plan, rs = build(zm, st, 0.0, device_step=device_step)
    moved = []
    for t, lr in enumerate((2e-3, 0.0, 2e-3)):
        rs.muon.lr, rs.muon.weight_decay = lr, 0.0
        before = [x.clone() for x in rs.master_tensors]
        rs.step([(0, plan.padded_numel, [to_dev_u16(r) for r in replicas(100 + t, plan)])])
        moved.append([not torch.equal(a, b) for a, b in zip(before, rs.master_tensors)])
    assert moved[0] == moved[2] == [True] * len(moved[0])
    assert moved[1] == [k not in MATRICES for k in range(len(moved[1]))]


def test_a_captured_step_beside_eager_ones(zm, st):
    """Captured with one rate on a side stream, then an eager step with another rate on the current one, then the replay:
    as the same steps all eager."""
    plan, eager = build(zm, st, 0.05, device_step=True)
    _, mixed = build(zm, st, 0.05, device_step=True)
    reps = [to_dev_u16(r) for r in replicas(100, plan)]
    window = [(0, plan.padded_numel, reps)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    eager.step(window)
    mixed.step(window, stream=side.cuda_stream)          # eager: builds the tables
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        mixed.adamw(stream=side.cuda_stream)
    for t, lr in enumerate((5e-4, 2e-3, 1e-3, 2e-3)):
        if t % 2 == 0:
            for rs in (eager, mixed):
                rs.muon.lr = lr
                rs._prepared("muon", None, lambda s, rs=rs: rs._muon_table().prepare_step(
                    clip_scale=rs.scale, stream=s, **rs.muon.as_kwargs()), tuple(rs.muon.as_kwargs().values()))()
            torch.cuda.synchronize()
        else:
            graph.replay()
            eager.muon.lr = lr
            eager.adamw()
            torch.cuda.synchronize()
        for k in MATRICES:
            assert torch.equal(eager.master_tensors[k], mixed.master_tensors[k]), (t, k)
