"""Tables and prepared calls hold the tensors whose addresses they carry, also when the caller empties the lists that
it passed (stand-ins for device tensors: no address is dereferenced)."""
import gc
import weakref

import pytest
import torch

from test_state8_abi_cpu import _Stand, _stands

HYPER = dict(lr=1e-3, beta1=0.9, beta2=0.999, eps=1e-8, weight_decay=0.01)


@pytest.fixture
def zb(monkeypatch):
    from zero_partitioned_mixed_partition_amd import _binding as b
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    monkeypatch.setattr(b, "_mt8_create", lambda *a: b.ZERO_OK)
    monkeypatch.setattr(b, "_mt_create", lambda *a: b.ZERO_OK)
    return b


def _lists8():
    return [[t] for t in _stands([0] * 7)]


def _lists32():
    return [[_Stand(300, size, 0, 0x1000000 * (k + 1))] for k, size in enumerate((4, 4, 4, 2, 2))]


def _alive_after_clearing(lists, make):
    refs = [weakref.ref(t) for x in lists for t in x]
    holder = make(lists)
    for x in lists:
        x.clear()
    gc.collect()
    return holder, [r() is not None for r in refs]


@pytest.mark.parametrize("form", ["table", "list", "32-bit table", "32-bit list"])
def test_lists_emptied_by_the_caller(zb, form):
    make = {"table": lambda x: zb.MultiTensor8Table(*x),
            "list": lambda x: zb.prepare_multi_tensor_adamw8_step(*x, stream=0, **HYPER),
            "32-bit table": lambda x: zb.MultiTensorTable(*x),
            "32-bit list": lambda x: zb.prepare_multi_tensor_adamw_step(*x, stream=0, clip_scale=None, **HYPER)}[form]
    holder, alive = _alive_after_clearing(_lists32() if "32" in form else _lists8(), make)
    assert all(alive) and holder is not None


FORMS = ["8-bit", "8-bit scheduled", "32-bit", "32-bit scheduled", "reduce", "gather", "flatten"]


@pytest.mark.parametrize("form", FORMS)
def test_plans_and_lists_of_prepared_calls(zb, form):
    """Replicas, shards and tensors in a list that the caller empties, and a plan that it drops."""
    plan = zb.zero_partition_plan([300], 1, 1)
    dropped = weakref.ref(plan)
    plans = [plan]
    del plan
    t = _stands([0] * 7)
    f32 = [_Stand(300, 4, 0, 0x20000000 + 0x1000 * k) for k in range(3)]

    class Schedule:
        handle = None

    def make(lists):
        (x,), p = lists, plans[0]
        return {"8-bit": lambda: zb.prepare_reduce_adamw8_step(p, 0, x, 0, 300, *t[:5], t[6], stream=0, **HYPER),
                "8-bit scheduled": lambda: zb.prepare_reduce_adamw8_step_scheduled(
                    p, 0, x, 0, 300, *t[:5], t[6], Schedule, stream=0),
                "32-bit": lambda: zb.prepare_reduce_adamw_step(p, 0, x, 0, 300, *f32, t[6], stream=0, **HYPER),
                "32-bit scheduled": lambda: zb.prepare_reduce_adamw_step_scheduled(
                    p, 0, x, 0, 300, *f32, t[6], Schedule, stream=0),
                "reduce": lambda: zb.prepare_grad_reduce_shard(p, 0, x, 0, 300, t[5], None, None, 0),
                "gather": lambda: zb.prepare_gather_params(p, x, [t[6]], 0),
                "flatten": lambda: zb.prepare_flatten_params(p, x, t[6], 0)}[form]()
    one = [[_Stand(300, 2, 0, 0x9000000)]]
    holder, alive = _alive_after_clearing(one, make)
    plans.clear()
    gc.collect()
    assert all(alive) and dropped() is not None and holder is not None
