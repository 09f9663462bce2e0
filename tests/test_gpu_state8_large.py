"""The 8-bit AdamW and its conversions past 2^32 elements and past one grid row:
the arrays are zeros but for windows around the borders, which are compared bit
for bit with the oracle's step on them (numbered from their place), and the rest
is counted to be zeros still."""
import numpy as np
import pytest
import torch

import oracle
from gpu_util import assert_bits_equal, dev, host_f32, needs_gpu, note, to_dev_f32, to_dev_u16
from oracle import state8
from test_gpu_state8 import HP, check, make_grad, make_state

pytestmark = [pytest.mark.gpu, needs_gpu]


@pytest.fixture(scope="module")
def zm():
    import zero_partitioned_mixed_partition_amd as m
    torch.cuda.set_device(0)
    return m


def _room(need):
    torch.cuda.empty_cache()
    free, _ = torch.cuda.mem_get_info()
    if free < need * 1.05 + (4 << 30):
        pytest.skip(f"needs {need / 1e9:.0f} GB of device memory, {free / 1e9:.0f} free")


def _zeros(n):
    nb = state8.n_blocks(n)
    f = torch.zeros(n, dtype=torch.float32, device=dev())
    b = [torch.zeros(k, dtype=torch.uint8, device=dev()) for k in (n, nb, n, nb)]
    h = [torch.zeros(n, dtype=torch.int16, device=dev()) for _ in range(2)]
    return [f] + b, h[0], h[1]


def _windows(n, borders):
    """Block-aligned windows of 1,280 elements (the last maybe shorter) around each border."""
    out = []
    for b in borders:
        lo = max(0, b // 128 * 128 - 640)
        out.append((lo, min(n, lo + 1280)))
    return out


def _fill(state, grad, windows):
    held = []
    for k, (a, b) in enumerate(windows):
        s, g = make_state(b - a, 500 + k), make_grad(b - a, 600 + k)
        for t, x in zip(state, s):
            lo = a // 128 if t.numel() < state[0].numel() else a
            t[lo:lo + len(x)] = torch.from_numpy(x).to(dev())
        grad[a:b] = to_dev_u16(g)
        held.append((s, g))
    return held


def _check_windows(state, out, held, windows, step, seed, first):
    for (a, b), (s, g) in zip(windows, held):
        note(f"window [{a}, {b})")
        want = oracle.adamw8_step(*s, g, step, seed=seed, first_element=first + a, **HP)
        got = [state[0][a:b], state[1][a:b], state[2][a // 128:-(-b // 128)], state[3][a:b],
               state[4][a // 128:-(-b // 128)], out[a:b]]
        check(got, want, f"window [{a}, {b})")
    inside = sum(int(torch.count_nonzero(out[a:b])) for a, b in windows)
    total = sum(int(torch.count_nonzero(c)) for c in out.split(1 << 30))
    assert total == inside, "a parameter outside the windows changed"
    for t in (state[1], state[3]):
        inside = sum(int(torch.count_nonzero(t[a:b])) for a, b in windows)
        assert sum(int(torch.count_nonzero(c)) for c in t.split(1 << 30)) == inside, "a code outside the windows changed"


@pytest.mark.parametrize("form", ["flat", "list", "table", "reduce"])
def test_steps_past_2_32_elements(zm, form):
    n = (1 << 32) + 128 * 9 + 37
    _room(n * 10 + n // 64)
    state, grad, out = _zeros(n)
    windows = _windows(n, [0, 1 << 31, 1 << 32, n])
    windows = windows[:2] + [(windows[2][0], n)]           # the last two meet
    held = _fill(state, grad, windows)
    first = 128 * 5
    note(f"{form}, {n} elements")
    if form == "flat":
        zm.zero_shard_adamw8_step(*state, grad, out, 3, seed=4, first_element=first, **HP)
    elif form == "list":
        zm.zero_multi_tensor_adamw8_step(*[[t] for t in state], [grad], [out], 3, seed=4, first_element=first, **HP)
    elif form == "table":
        zm.MultiTensor8Table(*[[t] for t in state], [grad], [out], first_element=first).step(3, seed=4, **HP)
    else:
        plan = zm.zero_partition_plan([n], 1, 1)
        zm.zero_reduce_adamw8_step(plan, 0, [grad], 0, n, *state, out, 3, seed=4, first_element=first, **HP)
    _check_windows(state, out, held, windows, 3, 4, first)


def test_flat_step_past_one_grid_row(zm):
    """More workgroups than one grid dimension holds (2^25 - 1 of 512 elements)."""
    row = ((1 << 25) - 1) * 512
    n = row + 128 * 21 + 11
    _room(n * 10 + n // 64)
    state, grad, out = _zeros(n)
    windows = _windows(n, [0, row // 2, row, n])
    windows = windows[:2] + [(windows[2][0], n)]
    held = _fill(state, grad, windows)
    note(f"{n} elements")
    zm.zero_shard_adamw8_step(*state, grad, out, 2, seed=9, **HP)
    _check_windows(state, out, held, windows, 2, 9, 0)


def test_conversions_past_2_32_elements(zm):
    n = (1 << 32) + 128 * 3 + 5
    nb = state8.n_blocks(n)
    _room(n * 5 + nb)
    x = torch.zeros(n, dtype=torch.float32, device=dev())
    codes, scales = torch.zeros(n, dtype=torch.uint8, device=dev()), torch.zeros(nb, dtype=torch.uint8, device=dev())
    windows = _windows(n, [0, 1 << 31])
    windows.append((n // 128 * 128 - 1280, n))
    rng = np.random.default_rng(7)
    held = []
    for a, b in windows:
        h = (rng.standard_normal(b - a) * 1e-3).astype(np.float32)
        x[a:b] = to_dev_f32(h)
        held.append(state8.encode(h, False))
    zm.zero_state8_quantize(x, codes, scales)
    for (a, b), (c, s) in zip(windows, held):
        assert_bits_equal(codes[a:b].cpu().numpy(), c, "codes")
        assert_bits_equal(scales[a // 128:-(-b // 128)].cpu().numpy(), s, "scales")
    assert sum(int(torch.count_nonzero(t)) for t in codes.split(1 << 30)) == sum(np.count_nonzero(c) for c, _ in held)
    x.fill_(5.0)
    zm.zero_state8_dequantize(codes, scales, x)
    for (a, b), (c, s) in zip(windows, held):
        assert_bits_equal(host_f32(x[a:b]).view(np.uint32), state8.decode(c, s).view(np.uint32), "values")
    assert sum(int(torch.count_nonzero(t)) for t in x.split(1 << 30)) == sum(
        np.count_nonzero(state8.decode(c, s)) for c, s in held)
