"""The order that a MuonTable gives the streams that share its workspace, with stand-ins for the streams (no GPU)."""
import pytest
import torch

from test_muon_held_cpu import HYPER, _stands, zb  # noqa: F401
from test_state8_abi_cpu import _Stand


class _Stream:
    def __init__(self, handle, log):
        self.cuda_stream, self.log = handle, log

    def wait_stream(self, other):
        self.log.append(("wait", self.cuda_stream, other.cuda_stream))


class _Workspace(_Stand):
    def __init__(self, log):
        super().__init__(1 << 20, 1, 0, 0x70000000)
        self.log = log

    def record_stream(self, stream):
        self.log.append(("record", stream.cuda_stream))


@pytest.fixture
def world(zb, monkeypatch):  # noqa: F811
    """The table, what happens in order, and the current stream and whether it is being captured (to be set)."""
    b, made, _ = zb
    out, now = [], {"current": 64, "capturing": False}
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: _Stream(now["current"], out))
    monkeypatch.setattr(torch.cuda, "default_stream", lambda device=None: _Stream(0, out))
    monkeypatch.setattr(torch.cuda, "ExternalStream", lambda handle, device=None: _Stream(handle, out))
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: now["capturing"])
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda index: now["current"], raising=False)
    monkeypatch.setattr(torch, "empty", lambda n, dtype, device: _Workspace(out))
    monkeypatch.setattr(b, "_muont_ws", lambda h: 1 << 20)
    return b.MuonTable(*[[t] for t in _stands()], [(20, 15)]), out, now


def test_each_further_stream_waits_for_the_one_that_made_the_workspace(world):
    table, log, now = world
    table.prepare_step(**HYPER)                          # on the current one; never called
    assert log == []
    table.prepare_step(stream=4096, **HYPER)
    assert log == [("wait", 4096, 64), ("record", 4096)]
    table.prepare_step(stream=0, **HYPER)
    assert log[2:] == [("wait", 0, 64), ("record", 0)]
    now["current"] = 128
    table.prepare_step(**HYPER)
    assert log[4:] == [("wait", 128, 64), ("record", 128)]
    for stream in (4096, 0, 128, 64, None):
        table.prepare_step(stream=stream, **HYPER)
    assert len(log) == 6


def test_made_for_a_side_stream(world):
    table, log, _ = world
    table.prepare_step(stream=4096, **HYPER)
    assert log == [("wait", 4096, 64), ("record", 4096)]
    table.prepare_step(stream=8192, **HYPER)
    assert log[2:] == [("wait", 8192, 64), ("record", 8192)]
    table.prepare_step(stream=4096, **HYPER)
    table.prepare_step(**HYPER)
    assert len(log) == 4


def test_a_captured_stream_waits_for_none(world):
    table, log, now = world
    table.prepare_step(**HYPER)
    now.update(current=256, capturing=True)
    table.prepare_step(**HYPER)
    assert log == []
    now.update(current=64, capturing=False)
    table.prepare_step(stream=256, **HYPER)              # and eagerly on it afterwards
    assert log == [("wait", 256, 64), ("record", 256)]


def test_a_workspace_of_the_callers_is_the_callers_to_order(world):
    table, log, _ = world
    given = _Stand(1 << 20, 1, 0, 0x60000000)
    for stream in (None, 4096, 0):
        table.prepare_step(stream=stream, workspace=given, **HYPER)
    assert log == []
