"""The 8-bit steps over the borders of the random words' windows (2^28 elements), where a workgroup's elements may
lie on both sides: every form bit for bit against the oracle."""
import numpy as np
import pytest
import torch

import oracle
from gpu_util import dev, needs_gpu, note, to_dev_u16
from test_gpu_state8 import HP, check, make_grad, make_state, to_dev

pytestmark = [pytest.mark.gpu, needs_gpu]


@pytest.fixture(scope="module")
def zm():
    import zero_partitioned_mixed_partition_amd as m
    torch.cuda.set_device(0)
    return m


@pytest.mark.parametrize("form", ["flat", "flat-scheduled", "list", "table", "table-scheduled", "reduce",
                                  "reduce-scheduled"])
@pytest.mark.parametrize("border", [1 << 28, 37 << 28, 1 << 40])
@pytest.mark.parametrize("before", [128, 256, 384, 512, 128 * 5])
def test_steps_across_a_window_border(zm, form, border, before):
    n = 128 * 12 + 77
    first = border - before
    note(f"{form}, {n} elements from {first}")
    state, g = make_state(n, 1), make_grad(n, 2)
    d, out, dg = to_dev(state), torch.zeros(n, dtype=torch.int16, device=dev()), to_dev_u16(g)
    step = 1 if "scheduled" in form else 6
    seed = (1 << 63) + 11
    sched = zm.AdamWSchedule(HP["lr"], HP["beta1"], HP["beta2"], HP["eps"], HP["weight_decay"])
    lists = [[x] for x in d] + [[dg], [out]]
    plan = zm.zero_partition_plan([n], 1, 1)
    if form == "flat":
        zm.zero_shard_adamw8_step(*d, dg, out, step, seed=seed, first_element=first, **HP)
    elif form == "flat-scheduled":
        zm.zero_shard_adamw8_step_scheduled(*d, dg, out, sched, seed=seed, first_element=first)
    elif form == "list":
        zm.zero_multi_tensor_adamw8_step(*lists, step, seed=seed, first_element=first, **HP)
    elif form == "table":
        zm.MultiTensor8Table(*lists, first_element=first).step(step, seed=seed, **HP)
    elif form == "table-scheduled":
        zm.MultiTensor8Table(*lists, first_element=first).step_scheduled(sched, seed=seed)
    elif form == "reduce":
        zm.zero_reduce_adamw8_step(plan, 0, [dg], 0, n, *d, out, step, seed=seed, first_element=first, **HP)
    else:
        zm.zero_reduce_adamw8_step_scheduled(plan, 0, [dg], 0, n, *d, out, sched, seed=seed, first_element=first)
    torch.cuda.synchronize()
    check(d + [out], oracle.adamw8_step(*state, g, step, seed=seed, first_element=first, **HP), form)


def test_list_tensors_on_both_sides_of_a_border(zm):
    """Ragged tensors numbered one after the other across a border, in the list and in the table."""
    numels = [100, 128, 1000, 1, 700, 64]
    states = [make_state(n, 20 + k) for k, n in enumerate(numels)]
    grads = [make_grad(n, 40 + k) for k, n in enumerate(numels)]
    first = (3 << 28) - 128 * 6
    for form in ("list", "table"):
        note(form)
        ds = [to_dev(s) for s in states]
        lists = [[d[k] for d in ds] for k in range(5)] + [[to_dev_u16(g) for g in grads],
                                                          [torch.zeros(n, dtype=torch.int16, device=dev())
                                                           for n in numels]]
        if form == "list":
            zm.zero_multi_tensor_adamw8_step(*lists, 2, seed=5, first_element=first, **HP)
        else:
            zm.MultiTensor8Table(*lists, first_element=first).step(2, seed=5, **HP)
        torch.cuda.synchronize()
        at = first
        for k, n in enumerate(numels):
            want = oracle.adamw8_step(*states[k], grads[k], 2, seed=5, first_element=at, **HP)
            check(ds[k] + [lists[6][k]], want, f"{form} tensor {k}")
            at += -(-n // 128) * 128
    assert np.sign(first - (3 << 28)) != np.sign(at - (3 << 28))
