"""The order that RankStep.load_moments and moments give a side stream, with stand-ins for the streams (no GPU)."""
import pytest
import torch

from zero_partitioned_mixed_partition_amd import step


class _Stream:
    def __init__(self, handle, log):
        self.cuda_stream, self.log = handle, log

    def wait_stream(self, other):
        self.log.append(("wait", self.cuda_stream, other.cuda_stream))


@pytest.fixture
def log(monkeypatch):
    """What happens, in order: waits, tensors recorded on a stream, conversions. The current stream is 64."""
    out = []
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: _Stream(64, out))
    monkeypatch.setattr(torch.cuda, "default_stream", lambda device=None: _Stream(0, out))
    monkeypatch.setattr(torch.cuda, "ExternalStream", lambda handle, device=None: _Stream(handle, out))
    monkeypatch.setattr(torch.Tensor, "record_stream",
                        lambda self, s: out.append(("record", s.cuda_stream, self.data_ptr())))
    monkeypatch.setattr(step.zb, "zero_state8_quantize",
                        lambda x, c, s, second, stream: out.append(("convert", stream, x.data_ptr())))
    monkeypatch.setattr(step.zb, "zero_state8_dequantize",
                        lambda c, s, x, stream: out.append(("convert", stream, x.data_ptr())))
    return out


def _rank_step(zm, per_param):
    plan = zm.zero_partition_plan([1000, 37, 500], 2, 128)
    return step.RankStep(plan, 0, 1, step.Hyper(), 0.0, torch.device("cpu"), state_bits=8, per_param=per_param)


@pytest.mark.parametrize("per_param", [False, True])
@pytest.mark.parametrize("handle", [4096, 0])
def test_a_side_stream_waits_and_keeps_the_tensors(log, per_param, handle):
    import zero_partitioned_mixed_partition_amd as zm
    rs = _rank_step(zm, per_param)
    m, v = rs.moments(stream=handle)
    for back in (False, True):
        if back:
            rs.load_moments(m, v, stream=handle)
        tensors = [x.data_ptr() for x in ([*m, *v] if per_param else [m, v])]
        assert log[0] == ("wait", handle, 64)
        assert sorted(log[1:1 + len(tensors)]) == sorted(("record", handle, p) for p in tensors)
        assert sorted(log[1 + len(tensors):]) == sorted(("convert", handle, p) for p in tensors)
        log.clear()


@pytest.mark.parametrize("handle", [None, 64])
def test_the_current_stream_needs_neither(log, handle):
    import zero_partitioned_mixed_partition_amd as zm
    rs = _rank_step(zm, False)
    m, v = rs.moments(stream=handle)
    rs.load_moments(m, v, stream=handle)
    assert [what for what, _, _ in log] == ["convert"] * 4


def test_lengths_and_devices_are_refused_before_anything_is_enqueued(log):
    import zero_partitioned_mixed_partition_amd as zm
    rs = _rank_step(zm, False)
    n = rs.plan.shard_numel
    with pytest.raises(ValueError, match="length"):
        rs.load_moments(torch.zeros(n), torch.zeros(n - 1), stream=4096)
    with pytest.raises(ValueError, match="device tensors"):
        rs.load_moments(torch.zeros(n), torch.zeros(n, device="meta"), stream=4096)
    assert log == []
