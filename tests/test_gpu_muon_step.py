"""RankStep with Muon on the GPU: reduce, clip, update and gather in a row, against the oracle's formulas around
zero_orthogonalize's own bits (whose precision test_gpu_muon.py holds): bit for bit."""
import numpy as np
import pytest
import torch

import oracle
from tests.gpu_util import dev, host_f32, host_u16, needs_gpu, to_dev_f32, to_dev_u16

pytestmark = [pytest.mark.gpu, needs_gpu]

SHAPES = [(100, 64), (64,), (60, 260), (1, 7), (300, 300), (33,)]
NUMELS = [int(np.prod(s)) for s in SHAPES]
MATRICES = {t: s for t, s in enumerate(SHAPES) if len(s) == 2}


@pytest.fixture(scope="module")
def zm():
    import zero_partitioned_mixed_partition_amd as m
    return m


@pytest.fixture(scope="module")
def st():
    from zero_partitioned_mixed_partition_amd import step as s
    return s


def masters(seed):
    rng = np.random.default_rng(seed)
    return [rng.normal(size=n).astype(np.float32) * 0.02 for n in NUMELS]


def replicas(seed, plan, n=2):
    rng = np.random.default_rng(seed)
    flat = np.zeros((n, plan.padded_numel), np.float32)
    flat[:, :sum(NUMELS)] = rng.normal(size=(n, sum(NUMELS))) * 1e-3
    return [oracle.f32_to_bf16(f) for f in flat]


def build(zm, st, max_norm=1.0, **kw):
    plan = zm.zero_partition_plan(NUMELS, 1, 128)
    rs = st.RankStep(plan, 0, 1, st.Hyper(lr=1e-3), max_norm, dev(), per_param=True,
                     muon=st.MuonHyper(lr=2e-3, momentum=0.9, weight_decay=0.1), muon_shapes=MATRICES, **kw)
    for x, m in zip(rs.master_tensors, masters(0)):
        x.copy_(to_dev_f32(m))
    return plan, rs


def expected(zm, plan, steps, max_norm=1.0):
    """The state after the steps: Muon's tensors through zero_orthogonalize, the rest through the oracle's AdamW."""
    ref = oracle.partition_plan(NUMELS, 1, 128)
    state = [{"p": m.copy(), "m": np.zeros_like(m), "v": np.zeros_like(m), "bits": None} for m in masters(0)]
    for t in range(steps):
        reps = replicas(100 + t, plan)
        grad = np.zeros(ref.shard_numel, np.uint16)
        oracle.reduce_shard(ref, 0, reps, 0, grad)
        clip = float(oracle.clip_scale([oracle.sqnorm(grad)], max_norm)) if max_norm > 0 else 1.0
        at = 0
        table = []
        for k, s in enumerate(state):
            g = grad[at:at + NUMELS[k]]
            at += NUMELS[k]
            if k in MATRICES:
                s["m"], u = oracle.muon.momentum(s["m"], g, 0.9, True, clip)
                table.append((k, u))
            else:
                s["p"], s["m"], s["v"], s["bits"] = oracle.adamw_step(s["p"], s["m"], s["v"], g, t + 1, clip=clip, lr=1e-3, beta1=0.9,
                                                                     beta2=0.999, eps=1e-8, weight_decay=0.01)
        # the list's orthogonalised updates: the table's step from zero weights at rate 1 is minus them
        mats = [to_dev_f32(np.zeros(len(u), np.float32)) for _, u in table]
        bufs = [to_dev_f32(u) for _, u in table]
        outs = [torch.zeros(len(u), dtype=torch.int16, device=dev()) for _, u in table]
        zeros = [torch.zeros(len(u), dtype=torch.int16, device=dev()) for _, u in table]
        # momentum just below 1 and no gradient: u = momentum * buffer in fp32, a power of two
        half = [b * 2 for b in bufs]
        zm.MuonTable(mats, half, zeros, outs, [MATRICES[k] for k, _ in table], [1.0] * len(table)).step(
            lr=1.0, momentum=0.5, nesterov=False)
        for (k, _), o in zip(table, outs):
            rows, cols = MATRICES[k]
            bits = host_u16(o) ^ 0x8000                  # p = 0 - o, exact in bf16
            s = state[k]
            s["p"], s["bits"] = oracle.muon.apply(s["p"], bits, 2e-3, zm.muon_scale(rows, cols), 0.1)
    return state


def check(rs, state):
    for k, s in enumerate(state):
        assert (host_f32(rs.master_tensors[k]).view(np.uint32) == s["p"].view(np.uint32)).all(), k
        assert (host_f32(rs.exp_avg_tensors[k]).view(np.uint32) == s["m"].view(np.uint32)).all(), k
        assert (host_u16(rs.tensors[k]) == s["bits"]).all(), k


@pytest.mark.parametrize("device_step", [False, True])
@pytest.mark.parametrize("max_norm", [0.0, 0.05])
def test_steps(zm, st, device_step, max_norm):
    plan, rs = build(zm, st, max_norm, device_step=device_step)
    for t in range(3):
        reps = [to_dev_u16(r) for r in replicas(100 + t, plan)]
        rs.step([(0, plan.padded_numel, reps)])
    check(rs, expected(zm, plan, 3, max_norm))
    assert rs.steps_applied() == 3


def test_a_step_with_a_non_finite_norm_changes_nothing(zm, st):
    plan, rs = build(zm, st)
    reps = [to_dev_u16(r) for r in replicas(100, plan)]
    rs.step([(0, plan.padded_numel, reps)])
    before = [x.clone() for x in rs.master_tensors + rs.exp_avg_tensors + rs.tensors]
    reps[0][5] = 0x7F80                                  # an infinity
    rs.step([(0, plan.padded_numel, reps)])
    for a, b in zip(before, rs.master_tensors + rs.exp_avg_tensors + rs.tensors):
        assert torch.equal(a, b)


def test_captured_step(zm, st):
    """The whole step in a graph, replayed with new gradients and eager work between: the eager steps."""
    plan, eager = build(zm, st, 0.05, device_step=True)
    _, graphed = build(zm, st, 0.05, device_step=True)
    reps = [[to_dev_u16(r) for r in replicas(100, plan)] for _ in range(2)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    eager.step([(0, plan.padded_numel, reps[0])])
    graphed.step([(0, plan.padded_numel, reps[1])], stream=side.cuda_stream)       # eager: builds the tables
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        graphed.step([(0, plan.padded_numel, reps[1])], stream=side.cuda_stream)
    for t in range(1, 4):
        for k in range(2):
            for d, r in zip(reps[k], replicas(100 + t, plan)):
                d.copy_(to_dev_u16(r))
        torch.cuda.synchronize()
        g.replay()
        eager.step([(0, plan.padded_numel, reps[0])])
        torch.cuda.synchronize()
        for a, b in zip(eager.master_tensors + eager.exp_avg_tensors + eager.tensors,
                        graphed.master_tensors + graphed.exp_avg_tensors + graphed.tensors):
            assert torch.equal(a, b), t
    assert graphed.steps_applied() == 4
