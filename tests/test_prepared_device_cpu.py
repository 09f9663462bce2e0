"""A prepared 8-bit call belongs to the device of its tensors: made while another device is current, it is refused (the
default stream's handle is the same on every device). Stand-ins for device tensors; no address is dereferenced."""
import pytest
import torch

from test_state8_abi_cpu import _Stand, _stands

HYPER = dict(lr=1e-3, beta1=0.9, beta2=0.999, eps=1e-8, weight_decay=0.01)


@pytest.mark.parametrize("form", ["step", "list", "reduce", "empty list"])
def test_prepared_calls_on_another_current_device(monkeypatch, form):
    from zero_partitioned_mixed_partition_amd import _binding as zb
    current, made = [0], []
    monkeypatch.setattr(torch.cuda, "current_device", lambda: current[0])
    for name in ("_adamw8", "_mt_adamw8", "_reduce_adamw8"):
        monkeypatch.setattr(zb, name, lambda *a: made.append(a) or zb.ZERO_OK)
    t = _stands([0] * 7)
    plan = zb.zero_partition_plan([300], 1, 1)
    call = {"step": lambda: zb.prepare_shard_adamw8_step(*t, stream=0, **HYPER),
            "list": lambda: zb.prepare_multi_tensor_adamw8_step(*[[x] for x in t], stream=0, **HYPER),
            "empty list": lambda: zb.prepare_multi_tensor_adamw8_step(*[[]] * 7, stream=0, **HYPER),
            "reduce": lambda: zb.prepare_reduce_adamw8_step(plan, 0, [_Stand(300, 2, 0, 0x9000000)], 0, 300, *t[:5],
                                                            t[6], stream=0, **HYPER)}[form]()
    call(1)
    current[0] = 1
    if form == "empty list":                        # touches no device
        call(2)
    else:
        with pytest.raises(ValueError, match="device 0, the current device is 1"):
            call(2)
        current[0] = 0
        call(2)
    assert len(made) == 2
