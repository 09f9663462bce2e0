"""RankStep.load_moments and moments on a side stream while the current stream is busy with memory that the calls'
tensors take over or leave behind: bit for bit against the oracle's conversions."""
import numpy as np
import pytest
import torch

from gpu_util import assert_bits_equal, dev, host_f32, needs_gpu, note, to_dev_f32
from oracle import state8

pytestmark = [pytest.mark.gpu, needs_gpu]

BUSY = 100_000_000        # cycles that a stream is held: some 50 ms


@pytest.fixture(scope="module")
def zm():
    import zero_partitioned_mixed_partition_amd as m
    torch.cuda.set_device(0)
    return m


def _rank_step(zm, per_param=False):
    from zero_partitioned_mixed_partition_amd.step import Hyper, RankStep
    plan = zm.zero_partition_plan([700_001, 37, 300_000], 2, 128)
    return RankStep(plan, 0, 1, Hyper(), 0.0, dev(), state_bits=8, per_param=per_param)


def _values(n, seed):
    rng = np.random.default_rng(seed)
    return (rng.standard_normal(n) * 1e-3).astype(np.float32), (rng.random(n) * 1e-6).astype(np.float32)


def _held(rs):
    torch.cuda.synchronize()
    return [t.cpu().numpy() for t in (rs.exp_avg, rs.exp_avg_scale, rs.exp_avg_sq, rs.exp_avg_sq_scale)]


@pytest.mark.parametrize("default_stream_is_side", [False, True])
def test_moments_on_a_side_stream(zm, default_stream_is_side):
    """The results take memory that a queued fill of the current stream still writes; then they are dropped while
    the side stream still has to write them, and the memory is filled again on the current stream."""
    rs = _rank_step(zm)
    n = rs.plan.shard_numel
    m, v = _values(n, 1)
    rs.load_moments(to_dev_f32(m), to_dev_f32(v))
    want = [state8.decode(*state8.encode(m, False)), state8.decode(*state8.encode(v, True))]
    current = torch.cuda.Stream() if default_stream_is_side else torch.cuda.current_stream()
    side = torch.cuda.default_stream() if default_stream_is_side else torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(current):
        junk = [torch.empty(n, device=dev()) for _ in range(2)]
        places = {x.data_ptr() for x in junk}
        torch.cuda._sleep(BUSY)
        for x in junk:
            x.fill_(7.0)
        del junk, x
        got = rs.moments(stream=side.cuda_stream)
        note(f"results in the freed memory: {sum(x.data_ptr() in places for x in got)} of 2")
        torch.cuda.synchronize()
        for g, w in zip(got, want):
            assert_bits_equal(host_f32(g).view(np.uint32), w.view(np.uint32), "moments")
        del got, g
        with torch.cuda.stream(side):
            torch.cuda._sleep(BUSY)
        rs.moments(stream=side.cuda_stream)          # dropped at once
        after = [torch.full((n,), 3.0, device=dev()) for _ in range(2)]
        torch.cuda.synchronize()
        assert all(bool((x == 3.0).all()) for x in after), "memory in use on the side stream was handed out"


def test_load_moments_on_a_side_stream(zm):
    """The given tensors are still to be computed on the current stream, and are dropped and their memory filled
    before the side stream has read them."""
    rs = _rank_step(zm)
    n = rs.plan.shard_numel
    m, v = _values(n, 2)
    dm, dv = to_dev_f32(m), to_dev_f32(v)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(2 * BUSY)
    torch.cuda._sleep(BUSY)
    x, y = dm * 1.0, dv * 1.0
    rs.load_moments(x, y, stream=side.cuda_stream)
    del x, y
    after = [torch.full((n,), 3.0, device=dev()) for _ in range(2)]
    got = _held(rs)
    want = [*state8.encode(m, False), *state8.encode(v, True)]
    for g, w, name in zip(got, want, ("exp_avg", "exp_avg_scale", "exp_avg_sq", "exp_avg_sq_scale")):
        assert_bits_equal(g, w, name)
    assert all(bool((t == 3.0).all()) for t in after)


def test_per_parameter_moments_on_a_side_stream(zm):
    rs = _rank_step(zm, per_param=True)
    lens = [ln for (_, _, _, ln) in rs.segments]
    given = [_values(k, 10 + i) for i, k in enumerate(lens)]
    side = torch.cuda.Stream()
    torch.cuda._sleep(BUSY)
    rs.load_moments([to_dev_f32(m) for m, _ in given], [to_dev_f32(v) for _, v in given], stream=side.cuda_stream)
    got = rs.moments(stream=side.cuda_stream)
    torch.cuda.synchronize()
    for (m, v), gm, gv in zip(given, *got):
        assert_bits_equal(host_f32(gm).view(np.uint32), state8.decode(*state8.encode(m, False)).view(np.uint32), "m")
        assert_bits_equal(host_f32(gv).view(np.uint32), state8.decode(*state8.encode(v, True)).view(np.uint32), "v")
