"""Which marshalled calls a RankStep keeps: those of other streams with the same buffers (a captured step reads their device
tables at every replay), and none that holds earlier buffers. No call reaches the device."""
import gc
import weakref

import pytest
import torch

from zero_partitioned_mixed_partition_amd import step


class _Call:
    def __call__(self):
        pass


@pytest.fixture
def rs(monkeypatch):
    import zero_partitioned_mixed_partition_amd as zm
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: type("S", (), {"cuda_stream": 64})())
    return step.RankStep(zm.zero_partition_plan([12, 5], 1, 1), 0, 1, step.Hyper(), 0.0, torch.device("cpu"))


def test_another_stream_leaves_the_call_of_the_first(rs):
    made = []

    def build(stream):
        made.append((stream, weakref.ref(call := _Call())))
        return call

    for sig in (None, ("buffers",)):
        made.clear()
        key = ("call", sig)
        for stream in (4096, None, 4096, 64, None, 8192):
            rs._prepared(key, stream, build, sig)()
        gc.collect()
        assert [s for s, _ in made] == [4096, 64, 8192]
        assert all(r() is not None for _, r in made)


def test_a_new_signature_releases_the_old_buffers_on_every_stream(rs):
    made = []

    def build(stream):
        made.append(weakref.ref(call := _Call()))
        return call

    for stream in (4096, 64, 8192):
        rs._prepared("call", stream, build, "first")()
    rs._prepared("call", 64, build, "second")()
    gc.collect()
    assert [r() is None for r in made] == [True, True, True, False]
    rs._prepared("call", 4096, build, "second")()
    gc.collect()
    assert made[3]() is not None and len(made) == 5
