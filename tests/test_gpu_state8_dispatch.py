"""Launch choices of the 8-bit steps that small single calls do not reach: a table's second launch, a list's batch
that ends before 48 tensors, the two-at-a-time reduce with more than four replicas, and the scheduled kernels at odd
addresses and with many replicas. Bit for bit against the oracle (large arrays on windows, see
test_gpu_state8_large)."""
import numpy as np
import pytest
import torch

import oracle
from gpu_util import assert_bits_equal, dev, host_u16, needs_gpu, note, to_dev_f32, to_dev_u16
from oracle import state8
from test_gpu_state8 import HP, check, make_grad, make_state, to_dev, u8
from test_gpu_state8_large import _check_windows, _fill, _room, _windows, _zeros

pytestmark = [pytest.mark.gpu, needs_gpu]

TABLE_LAUNCH = ((1 << 32) // 256 - 1) // 8 * 8       # workgroups of 512 elements in a table's launch
LIST_LAUNCH = (1 << 25) - 1                          # and at most in a list's


@pytest.fixture(scope="module")
def zm():
    import zero_partitioned_mixed_partition_amd as m
    torch.cuda.set_device(0)
    return m


def _cut(state, grad, out, cuts):
    """The arrays as a list of tensors with the given borders (multiples of 128 but for the last)."""
    sl = list(zip(cuts, cuts[1:]))
    parts = [[t[a:b] for a, b in sl] if k in (0, 1, 3) else [t[a // 128:-(-b // 128)] for a, b in sl]
             for k, t in enumerate(state)]
    return parts + [[grad[a:b] for a, b in sl], [out[a:b] for a, b in sl]]


def test_a_table_of_two_launches(zm):
    """Four tensors over a little more than 2^24 workgroups: the border between the launches lies inside the third."""
    edge = TABLE_LAUNCH * 512
    n = edge + 512 * 21 + 128 * 3 + 77
    _room(n * 10 + n // 64)
    state, grad, out = _zeros(n)
    cuts = [0, 512 * 1000, edge // 2, edge + 512 * 9, n]
    windows = _windows(n, [0, cuts[1], cuts[2], edge, n])
    windows[-1] = (windows[3][1], n)
    held = _fill(state, grad, windows)
    table = zm.MultiTensor8Table(*_cut(state, grad, out, cuts), first_element=1280)
    assert table.blocks == -(-n // 512) and table.blocks > TABLE_LAUNCH
    note(f"{table.blocks} workgroups")
    table.step(3, seed=4, **HP)
    torch.cuda.synchronize()
    _check_windows(state, out, held, windows, 3, 4, 1280)


def test_a_list_batch_that_ends_early(zm):
    """Two tensors that do not fit one launch together, and a small one that joins the second."""
    size = 512 * (LIST_LAUNCH // 2 + 2)
    sizes = [size, size, 128 * 9 + 5]
    n = sum(sizes)
    _room(n * 10 + n // 64)
    state, grad, out = _zeros(n)
    cuts = [0, size, 2 * size, n]
    windows = _windows(n, [0, size, 2 * size])
    windows[-1] = (windows[-1][0], n)
    held = _fill(state, grad, windows)
    note(f"{n} elements in {len(sizes)} tensors of {sizes}")
    zm.zero_multi_tensor_adamw8_step(*_cut(state, grad, out, cuts), 2, seed=9, first_element=0, **HP)
    torch.cuda.synchronize()
    _check_windows(state, out, held, windows, 2, 9, 0)


@pytest.mark.parametrize("R", [5, 8, 9])
@pytest.mark.parametrize("off", [0, 1])
def test_reduce_of_many_replicas_on_a_large_window(zm, R, off):
    """Past 2^22 elements two replicas are loaded at a time, at odd addresses one."""
    n = (1 << 22) + 131
    note(f"{R} replicas of {n}, off {off}")
    plan, ref = zm.zero_partition_plan([n], 1, 1), oracle.partition_plan([n], 1, 1)
    reps = [make_grad(n, 300 + k) for k in range(R)]
    state = make_state(n, 310)
    d, out = to_dev(state), torch.zeros(n, dtype=torch.int16, device=dev())
    d_reps = [torch.cat([torch.zeros(off, dtype=torch.int16, device=dev()), to_dev_u16(r)])[off:] for r in reps]
    grad_out = torch.zeros(n, dtype=torch.int16, device=dev())
    g = np.zeros(n, np.uint16)
    oracle.reduce_shard(ref, 0, reps, 0, g)
    zm.zero_reduce_adamw8_step(plan, 0, d_reps, 0, n, *d, out, 4, seed=6, shard_grad=grad_out, **HP)
    torch.cuda.synchronize()
    assert_bits_equal(host_u16(grad_out), g, "averaged gradient")
    check(d + [out], oracle.adamw8_step(*state, g, 4, seed=6, **HP), "one pass")


@pytest.mark.parametrize("form,R,off", [("flat", 1, 1), ("flat", 1, 3), ("table", 1, 1), ("reduce", 8, 0),
                                        ("reduce", 8, 1), ("reduce", 64, 0), ("reduce", 3, 0)])
def test_scheduled_steps_at_odd_addresses_and_with_many_replicas(zm, form, R, off):
    """Two scheduled steps with the advance between them, every array `off` elements into its allocation."""
    n = 128 * 61 + 45
    note(f"{form}, {R} replicas, off {off}")
    state = make_state(n, 320)
    f32 = torch.cat([torch.zeros(off, device=dev()), to_dev_f32(state[0])])[off:]
    d = [f32] + [u8(a, off) for a in state[1:]]
    out = torch.zeros(n + off, dtype=torch.int16, device=dev())[off:]
    reps = [torch.zeros(n + off, dtype=torch.int16, device=dev())[off:] for _ in range(R)]
    plan, ref = zm.zero_partition_plan([n], 1, 1), oracle.partition_plan([n], 1, 1)
    sched = zm.AdamWSchedule(HP["lr"], HP["beta1"], HP["beta2"], HP["eps"], HP["weight_decay"])
    table = zm.MultiTensor8Table(*[[x] for x in d], [reps[0]], [out], first_element=128) if form == "table" else None
    for t in (1, 2):
        host = [make_grad(n, 330 + 100 * t + k) for k in range(R)]
        for x, h in zip(reps, host):
            x.copy_(to_dev_u16(h))
        g = np.zeros(n, np.uint16)
        oracle.reduce_shard(ref, 0, host, 0, g)
        if form == "flat":
            zm.zero_shard_adamw8_step_scheduled(*d, reps[0], out, sched, seed=2, first_element=128)
        elif form == "table":
            table.step_scheduled(sched, seed=2)
        else:
            zm.zero_reduce_adamw8_step_scheduled(plan, 0, reps, 0, n, *d, out, sched, seed=2, first_element=128)
        sched.advance()
        torch.cuda.synchronize()
        want = oracle.adamw8_step(*state, g, t, seed=2, first_element=128, **HP)
        check(d + [out], want, f"step {t}")
        state = list(want[:5])
    assert sched.applied() == 2 and state8.n_blocks(n) == len(state[2])
