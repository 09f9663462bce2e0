"""Muon's tables and prepared calls hold the tensors whose addresses they carry, and belong to one device (stand-ins for
device tensors: no address is dereferenced)."""
import gc
import weakref

import pytest
import torch

from test_state8_abi_cpu import _Stand

HYPER = dict(lr=1e-3, momentum=0.95, weight_decay=0.1)


@pytest.fixture
def zb(monkeypatch):
    from zero_partitioned_mixed_partition_amd import _binding as b
    current = [0]
    monkeypatch.setattr(torch.cuda, "current_device", lambda: current[0])
    monkeypatch.setattr(b, "_muont_create", lambda *a: b.ZERO_OK)
    monkeypatch.setattr(b, "_muont_count", lambda h: 1)
    b_made = []
    monkeypatch.setattr(b, "_muon", lambda *a: b_made.append(a) or b.ZERO_OK)
    monkeypatch.setattr(b, "_muont_step", lambda *a: b_made.append(a) or b.ZERO_OK)
    b_made_and_current = (b, b_made, current)
    return b_made_and_current


def _arrays(device=0):
    return [_Stand(300, size, device, 0x1000000 * (k + 1)) for k, size in enumerate((4, 4, 2, 2))]


def _stands():
    s = _arrays()
    for t in s:
        t.dtype = torch.float32 if t.size == 4 else torch.bfloat16
    return s


def _workspace(device=0):
    return _Stand(1 << 30, 1, device, 0x70000000)


def test_a_table_holds_its_tensors(zb):
    b, made, _ = zb
    lists = [[t] for t in _stands()]
    clip = _Stand(1, 4, 0, 0x9000000)
    refs = [weakref.ref(x[0]) for x in lists] + [weakref.ref(clip)]
    table = b.MuonTable(*lists, [(20, 15)])
    prepared = table.prepare_step(clip_scale=clip, workspace=_workspace(), stream=0, **HYPER)
    for x in lists:
        x.clear()
    del clip, table
    gc.collect()
    assert all(r() is not None for r in refs)
    prepared()
    assert len(made) == 1
    del prepared
    gc.collect()
    assert not any(r() is not None for r in refs)


def test_a_prepared_step_holds_its_tensors(zb):
    b, made, _ = zb
    arrays, ws = _stands(), _workspace()
    refs = [weakref.ref(t) for t in arrays + [ws]]
    prepared = b.prepare_muon_step(*arrays, 20, 15, workspace=ws, stream=0, **HYPER)
    arrays.clear()
    del ws
    gc.collect()
    assert all(r() is not None for r in refs)
    prepared()
    assert len(made) == 1


def test_a_prepared_step_on_another_current_device(zb):
    b, made, current = zb
    prepared = b.prepare_muon_step(*_stands(), 20, 15, workspace=_workspace(), stream=0, **HYPER)
    current[0] = 1
    with pytest.raises(ValueError, match="device 0, the current device is 1"):
        prepared()
    current[0] = 0
    prepared()
    assert len(made) == 1


def test_tensors_of_another_device(zb):
    b, made, _ = zb
    for k in range(1, 4):
        arrays = _stands()
        arrays[k].dev = 1
        arrays[k].device = torch.device("cuda", 1)
        with pytest.raises(ValueError):
            b.prepare_muon_step(*arrays, 20, 15, workspace=_workspace(), stream=0, **HYPER)
        with pytest.raises(ValueError):
            b.MuonTable(*[[t] for t in arrays], [(20, 15)])
    with pytest.raises(ValueError):
        b.prepare_muon_step(*_stands(), 20, 15, workspace=_workspace(1), stream=0, **HYPER)
    with pytest.raises(ValueError):
        b.MuonTable(*[[t] for t in _stands()], [(20, 15)]).prepare_step(workspace=_workspace(1), stream=0, **HYPER)
    assert not made
