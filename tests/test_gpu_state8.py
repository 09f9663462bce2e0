"""AdamW with 8-bit moments on the GPU, bit for bit against the oracle: the flat
step, the table of many tensors, the reduce and update in one pass, the
conversions, their captured forms, and RankStep(state_bits=8).

Every operation of the step is one IEEE fp32 operation or an integer one, so
codes, scales and parameters are compared as bits; a NaN only has to meet a NaN
in the master weights (its payload is not specified)."""
import math

import numpy as np
import pytest
import torch

import oracle
import synth
from gpu_util import assert_bits_equal, dev, host_f32, host_u16, needs_gpu, note, to_dev_f32, to_dev_u16
from oracle import state8

pytestmark = [pytest.mark.gpu, needs_gpu]

HP = dict(lr=1e-3, beta1=0.9, beta2=0.999, eps=1e-8, weight_decay=0.01)
NAMES = ("master", "exp_avg", "exp_avg_scale", "exp_avg_sq", "exp_avg_sq_scale", "param")


@pytest.fixture(scope="module")
def zm():
    import zero_partitioned_mixed_partition_amd as m
    torch.cuda.set_device(0)
    return m


def u8(a, offset=0):
    """A device copy of bytes, `offset` bytes into its own allocation."""
    t = torch.empty(len(a) + offset, dtype=torch.uint8, device=dev())[offset:]
    t.copy_(torch.from_numpy(np.ascontiguousarray(a, dtype=np.uint8)))
    return t


def make_state(n, seed, spread=3.0):
    """master, codes and scales of a run in progress, with block sizes spread over e^spread."""
    rng = np.random.default_rng(seed)
    size = np.repeat(np.exp(rng.standard_normal(state8.n_blocks(n)) * spread) * 1e-3, 128)[:n]
    p = (rng.standard_normal(n) * 0.02).astype(np.float32)
    m, ms = state8.encode((rng.standard_normal(n) * size).astype(np.float32), False)
    v, vs = state8.encode((rng.random(n) * size * size).astype(np.float32), True)
    return [p, m, ms, v, vs]


def make_grad(n, seed, scale=1e-3):
    rng = np.random.default_rng(seed)
    return oracle.f32_to_bf16((rng.standard_normal(n) * scale).astype(np.float32))


def to_dev(state):
    return [to_dev_f32(state[0])] + [u8(a) for a in state[1:]]


def check(got, want, what):
    """got: device master, codes, scales, codes, scales, param; want: the oracle's arrays."""
    for name, g, w in zip(NAMES, got, want):
        g = g.cpu().numpy()
        if name == "master":
            nan = np.isnan(w)
            assert (np.isnan(g) == nan).all(), f"{what}: NaN places of the master weights"
            g, w = g.view(np.uint32).copy(), np.asarray(w, np.float32).view(np.uint32).copy()
            g[nan] = w[nan] = 0
        elif name == "param":
            g = g.view(np.uint16)
            nan = (w & 0x7FFF) > 0x7F80
            assert (((g & 0x7FFF) > 0x7F80) == nan).all(), f"{what}: NaN places of the parameters"
            g, w = g.copy(), w.copy()
            g[nan] = w[nan] = 0
        assert_bits_equal(g, w, f"{what}: {name}")


@pytest.mark.parametrize("n", [1, 3, 7, 8, 9, 127, 128, 129, 1000, 2047, 2048, 2049, 100_003, (1 << 20) + 5])
def test_flat_step_matches_oracle(zm, n):
    note(f"flat step n={n}")
    state = make_state(n, n)
    d = to_dev(state)
    out = torch.zeros(n, dtype=torch.int16, device=dev())
    clip = torch.full((1,), 0.5, device=dev())
    for t in (1, 2, 3):
        g = make_grad(n, 100 + t)
        zm.zero_shard_adamw8_step(*d, to_dev_u16(g), out, t, seed=77, first_element=1280, clip_scale=clip, **HP)
        want = oracle.adamw8_step(*state, g, t, seed=77, first_element=1280, clip=0.5, **HP)
        check(d + [out], want, f"n {n} step {t}")
        state = list(want[:5])


def test_flat_step_from_cleared_state(zm):
    n = 5000
    state = [np.zeros(n, np.float32)] + [np.zeros(k, np.uint8) for k in (n, state8.n_blocks(n)) * 2]
    d, out = to_dev(state), torch.zeros(n, dtype=torch.int16, device=dev())
    g = make_grad(n, 5)
    g[::3] = 0
    g[256:512] = 0                                    # two blocks that stay zero
    zm.zero_shard_adamw8_step(*d, to_dev_u16(g), out, 1, seed=1, **HP)
    want = oracle.adamw8_step(*state, g, 1, seed=1, **HP)
    check(d + [out], want, "first step")
    assert (want[2][2:4] == 0).all() and (want[4][2:4] == 0).all()


@pytest.mark.parametrize("offsets", [(1, 0, 0, 0, 0), (0, 1, 0, 0, 0), (0, 0, 3, 0, 0), (0, 0, 0, 1, 0), (0, 0, 0, 0, 1),
                                     (3, 5, 7, 1, 3), (2, 4, 4, 2, 4)])
def test_any_alignment(zm, offsets):
    """Arrays at element offsets (master, m, v, grad, param) of their allocations; the scales at odd bytes.
    The bytes around every written array stay as they were."""
    n = 128 * 37 + 77
    note(f"offsets {offsets}")
    state, g = make_state(n, 9), make_grad(n, 10)
    nb = state8.n_blocks(n)
    bufs = []

    def place(a, dtype, off):
        buf = torch.full(((len(a) + off) + 64,), 85, dtype=dtype, device=dev())
        view = buf[off:off + len(a)]
        view.copy_(torch.from_numpy(a.view(np.int16) if a.dtype == np.uint16 else a))
        bufs.append((buf, off, len(a)))
        return view

    p = place(state[0], torch.float32, offsets[0])
    m, ms = place(state[1], torch.uint8, offsets[1]), place(state[2], torch.uint8, 1)
    v, vs = place(state[3], torch.uint8, offsets[2]), place(state[4], torch.uint8, 3)
    o = place(np.zeros(n, np.uint16), torch.int16, offsets[4])
    dg = place(g, torch.int16, offsets[3])
    assert ms.numel() == nb
    zm.zero_shard_adamw8_step(p, m, ms, v, vs, dg, o, 4, seed=3, **HP)
    check([p, m, ms, v, vs, o], oracle.adamw8_step(*state, g, 4, seed=3, **HP), f"offsets {offsets}")
    for buf, off, k in bufs:
        rest = torch.cat([buf[:off], buf[off + k:]])
        assert (rest == 85).all(), "a byte outside the arrays changed"


def test_every_code_and_scale_as_input(zm):
    """Random codes of both signs (NaN codes among them) under every scale byte, with gradients that match, dwarf
    and vanish beside them."""
    rng = np.random.default_rng(3)
    n = 256 * 128
    p = rng.standard_normal(n).astype(np.float32)
    m = rng.integers(0, 256, n).astype(np.uint8)
    m[rng.random(n) < 0.9] &= 0xF7                     # most blocks without a NaN code
    m[: n // 2][(m[: n // 2] & 0x7F) == 0x7F] = 0
    v = rng.integers(0, 0x7F, n).astype(np.uint8)
    ms, vs = np.arange(256).astype(np.uint8), rng.permutation(256).astype(np.uint8)
    state = [p, m, ms, v, vs]
    for scale in (1e-20, 1.0, 1e18):
        note(f"gradients of size {scale}")
        d, out = to_dev(state), torch.zeros(n, dtype=torch.int16, device=dev())
        g = make_grad(n, 4, scale)
        zm.zero_shard_adamw8_step(*d, to_dev_u16(g), out, 2, seed=5, **HP)
        check(d + [out], oracle.adamw8_step(*state, g, 2, seed=5, **HP), f"gradients {scale}")


@pytest.mark.parametrize("coef", [1.0, 0.7312345, 3.0e-5])
def test_encoding_over_every_exponent(zm, coef):
    """With both betas 0 the moments are g and g^2 of the clipped gradient: 2^20 elements whose exponents spread over
    60 binades below their block's largest and whose blocks lie anywhere in bf16's range (some blocks subnormal,
    some with squares that overflow), so that every normal and subnormal code is met, and cut to zero."""
    rng = np.random.default_rng(11)
    n = 1 << 20
    sign, mant = rng.integers(0, 2, n), rng.integers(0, 128, n)
    top = np.repeat(rng.integers(1, 255, n // 128), 128)
    expo = np.maximum(top - rng.integers(0, 60, n) * (rng.random(n) < 0.9), 0)
    g = (sign << 15 | expo << 7 | mant).astype(np.uint16)
    state = [np.zeros(n, np.float32)] + [np.zeros(k, np.uint8) for k in (n, n // 128) * 2]
    hp = dict(HP, beta1=0.0, beta2=0.0)
    clip = torch.full((1,), coef, dtype=torch.float32, device=dev())
    d, out = to_dev(state), torch.zeros(n, dtype=torch.int16, device=dev())
    zm.zero_shard_adamw8_step(*d, to_dev_u16(g), out, 1, seed=13, clip_scale=clip, **hp)
    want = oracle.adamw8_step(*state, g, 1, seed=13, clip=np.float32(coef), **hp)
    check(d + [out], want, f"coefficient {coef}")
    seen = np.bincount(want[1] & 0x7F, minlength=128)
    note(f"codes of the first moment met: {np.count_nonzero(seen)}")
    assert (seen[:0x70] > 0).all()                      # every code below the top binade, whose share a coefficient sets


def test_non_finite_gradients_make_their_blocks_nan(zm):
    n = 128 * 6 + 5
    state, g = make_state(n, 12), make_grad(n, 13)
    for at, bits in ((5, 0x7F80), (300, 0xFF80), (301, 0x7FC0), (600, 0x7F7F), (n - 1, 0xFFC1)):
        g[at] = bits                                   # inf, -inf, NaN, the largest bf16 (its square overflows), NaN
    d, out = to_dev(state), torch.zeros(n, dtype=torch.int16, device=dev())
    for t in (1, 2):
        want = oracle.adamw8_step(*state, g, t, seed=2, **HP)
        zm.zero_shard_adamw8_step(*d, to_dev_u16(g), out, t, seed=2, **HP)
        check(d + [out], want, f"step {t}")
        state = list(want[:5])
        g = make_grad(n, 14)
    assert list(np.flatnonzero(want[4] == 255)) == [0, 2, 4, 6] and list(np.flatnonzero(want[2] == 255)) == [0, 2, 6]


@pytest.mark.parametrize("coef", [float("nan"), float("inf"), float("-inf")])
def test_non_finite_clip_skips(zm, coef):
    n = 3000
    state, g = make_state(n, 15), make_grad(n, 16)
    clip = torch.full((1,), coef, device=dev())
    d, out = to_dev(state), torch.full((n,), 7, dtype=torch.int16, device=dev())
    zm.zero_shard_adamw8_step(*d, to_dev_u16(g), out, 1, clip_scale=clip, **HP)
    table = zm.MultiTensor8Table(*[[x] for x in d], [to_dev_u16(g)], [out])
    table.step(1, clip_scale=clip, **HP)
    zm.zero_multi_tensor_adamw8_step(*[[x] for x in d], [to_dev_u16(g)], [out], 1, clip_scale=clip, **HP)
    plan = zm.zero_partition_plan([n], 1, 1)
    grad_out = torch.zeros(n, dtype=torch.int16, device=dev())
    zm.zero_reduce_adamw8_step(plan, 0, [to_dev_u16(g)], 0, n, *d, out, 1, clip_scale=clip, shard_grad=grad_out, **HP)
    check(d + [out], state + [np.full(n, 7, np.uint16)], "skipped")
    assert_bits_equal(host_u16(grad_out), g, "the reduce's gradient is still written")


def test_windows_and_far_elements_round_as_the_whole(zm):
    """The shard in three windows against the whole, numbered from past 2^35 (the words' high half)."""
    n = 128 * 50 + 3
    state, g = make_state(n, 17), make_grad(n, 18)
    first = (1 << 35) + 128 * 7
    d, out = to_dev(state), torch.zeros(n, dtype=torch.int16, device=dev())
    dg = to_dev_u16(g)
    for a, b in ((0, 128), (128, 128 * 33), (128 * 33, n)):
        zm.zero_shard_adamw8_step(d[0][a:b], d[1][a:b], d[2][a // 128:], d[3][a:b], d[4][a // 128:], dg[a:b], out[a:b], 6,
                                  seed=(1 << 64) - 1, first_element=first + a, **HP)
    check(d + [out], oracle.adamw8_step(*state, g, 6, seed=(1 << 64) - 1, first_element=first, **HP), "windows")


@pytest.mark.parametrize("case", ["beta1-0", "beta2-0", "betas-0", "lr-0", "wd", "eps", "late"])
def test_hyperparameter_corners(zm, case):
    hp = dict(HP, **{"beta1-0": dict(beta1=0.0), "beta2-0": dict(beta2=0.0), "betas-0": dict(beta1=0.0, beta2=0.0),
                     "lr-0": dict(lr=0.0), "wd": dict(weight_decay=5.0, lr=0.5), "eps": dict(eps=1.0),
                     "late": dict()}[case])
    step = 10 ** 9 if case == "late" else 3
    n = 4096
    state, g = make_state(n, 20), make_grad(n, 21)
    d, out = to_dev(state), torch.zeros(n, dtype=torch.int16, device=dev())
    zm.zero_shard_adamw8_step(*d, to_dev_u16(g), out, step, seed=9, **hp)
    check(d + [out], oracle.adamw8_step(*state, g, step, seed=9, **hp), case)


def _ragged(zm, seed, misaligned):
    rng = np.random.default_rng(seed)
    numels = [int(x) for x in np.exp(rng.uniform(0, np.log(20000), 70))] + [0, 1, 128, 129, 2048, 2049, 4096]
    states = [make_state(n, 1000 + k) if n else [np.zeros(0, np.float32)] + [np.zeros(0, np.uint8)] * 4
              for k, n in enumerate(numels)]
    grads = [make_grad(n, 2000 + k) for k, n in enumerate(numels)]
    lists = [[] for _ in range(7)]
    for k, (s, g) in enumerate(zip(states, grads)):
        off = k % 4 if misaligned else 0
        arrays = [torch.cat([torch.zeros(off, device=dev()), to_dev_f32(s[0])])[off:]]
        arrays += [u8(a, off) for a in s[1:]]
        arrays += [torch.cat([torch.zeros(off, dtype=torch.int16, device=dev()), to_dev_u16(g)])[off:],
                   torch.zeros(len(g), dtype=torch.int16, device=dev())]
        for lst, a in zip(lists, arrays):
            lst.append(a)
    return numels, states, grads, lists


@pytest.mark.parametrize("form", ["list", "table"])
@pytest.mark.parametrize("misaligned", [False, True])
def test_many_tensors_match_oracle_per_tensor(zm, misaligned, form):
    numels, states, grads, lists = _ragged(zm, 30, misaligned)
    table = zm.MultiTensor8Table(*lists, first_element=256)
    assert table.blocks == sum(-(-n // 512) for n in numels)
    clip = torch.full((1,), 0.25, device=dev())
    for t in (1, 2):
        if form == "table":
            table.step(t, seed=11, clip_scale=clip, **HP)
        else:
            zm.zero_multi_tensor_adamw8_step(*lists, t, seed=11, first_element=256, clip_scale=clip, **HP)
        first = 256
        for k, n in enumerate(numels):
            if n == 0:
                continue
            want = oracle.adamw8_step(*states[k], grads[k], t, seed=11, first_element=first, clip=0.25, **HP)
            check([lists[j][k] for j in (0, 1, 2, 3, 4, 6)], want, f"tensor {k} of {n}, step {t}")
            states[k] = list(want[:5])
            first += -(-n // 128) * 128


def test_table_equals_the_flat_step_on_views(zm):
    """Tensors of whole blocks cut from one shard: the flat step's bits."""
    n = 128 * 300
    state, g = make_state(n, 31), make_grad(n, 32)
    a, b = to_dev(state), to_dev(state)
    oa, ob = (torch.zeros(n, dtype=torch.int16, device=dev()) for _ in range(2))
    dg = to_dev_u16(g)
    cuts = [0, 128, 128 * 17, 128 * 200, n]
    sl = list(zip(cuts, cuts[1:]))
    table = zm.MultiTensor8Table(*[[t[x // s:y // s] for x, y in sl] for t, s in zip(b, (1, 1, 128, 1, 128))],
                                 [dg[x:y] for x, y in sl], [ob[x:y] for x, y in sl], first_element=1280)
    for t in (1, 2):
        zm.zero_shard_adamw8_step(*a, dg, oa, t, seed=4, first_element=1280, **HP)
        table.step(t, seed=4, **HP)
    for x, y in zip(a + [oa], b + [ob]):
        assert torch.equal(x, y)


def test_empty_table(zm):
    table = zm.MultiTensor8Table([], [], [], [], [], [], [])
    assert table.blocks == 0
    table.step(1, **HP)
    zm.zero_multi_tensor_adamw8_step([], [], [], [], [], [], [], 1, **HP)


@pytest.mark.parametrize("R,numels,n_ranks,align,rank,window,off", [
    (1, [5000], 1, 128, 0, None, 0), (2, [999, 2000, 31], 2, 128, 1, None, 0), (3, [70_001], 3, 1, 1, None, 0),
    (8, [70_001], 2, 128, 0, None, 0), (9, [70_001], 2, 128, 1, None, 0), (64, [9001], 1, 128, 0, None, 0),
    (8, [70_001], 2, 128, 1, (35_072, 12_800), 0), (8, [70_001], 2, 128, 1, (20_000, 50_144), 0),
    (5, [70_001], 2, 128, 1, None, 1)])
def test_reduce_step_matches_oracle_and_the_two_calls(zm, R, numels, n_ranks, align, rank, window, off):
    plan = zm.zero_partition_plan(numels, n_ranks, align)
    ref = oracle.partition_plan(numels, n_ranks, align)
    P, S = ref.padded_numel, ref.shard_numel
    begin, count = window or (0, P)
    note(f"R={R} S={S} window {begin}+{count} off {off}")
    reps = [make_grad(P, 40 + k) for k in range(R)]
    state = make_state(S, 41)
    first = rank * state8.n_blocks(S) * 128
    d_reps = [torch.cat([torch.zeros(off, dtype=torch.int16, device=dev()), to_dev_u16(r[begin:begin + count])])[off:]
              for r in reps]
    lo, hi = max(begin - rank * S, 0), min(begin + count - rank * S, S)
    g = np.zeros(S, np.uint16)
    oracle.reduce_shard(ref, rank, [r[begin:begin + count] for r in reps], begin, g)
    b0, b1 = lo // 128, -(-hi // 128)
    part = [state[0][lo:hi], state[1][lo:hi], state[2][b0:b1], state[3][lo:hi], state[4][b0:b1]]
    res = oracle.adamw8_step(*part, g[lo:hi], 5, seed=6, first_element=first + lo, **HP)
    want = [x.copy() for x in state] + [np.full(S, 3, np.uint16)]
    for k, (x, y) in enumerate(((lo, hi), (lo, hi), (b0, b1), (lo, hi), (b0, b1), (lo, hi))):
        want[k][x:y] = res[k]
    for with_grad in (False, True):
        d, out = to_dev(state), torch.full((S,), 3, dtype=torch.int16, device=dev())
        grad_out = torch.full((S,), 9, dtype=torch.int16, device=dev()) if with_grad else None
        zm.zero_reduce_adamw8_step(plan, rank, d_reps, begin, count, *d, out, 5, seed=6, first_element=first,
                                   shard_grad=grad_out, **HP)
        check(d + [out], want, f"one pass, gradient {with_grad}")
        if with_grad:
            w = np.full(S, 9, np.uint16)
            w[lo:hi] = g[lo:hi]
            assert_bits_equal(host_u16(grad_out), w, "averaged gradient")
    d, out = to_dev(state), torch.full((S,), 3, dtype=torch.int16, device=dev())
    dg = torch.zeros(S, dtype=torch.int16, device=dev())
    zm.zero_grad_reduce_shard(plan, rank, d_reps, begin, count, dg)
    zm.zero_shard_adamw8_step(d[0][lo:hi], d[1][lo:hi], d[2][b0:b1], d[3][lo:hi], d[4][b0:b1], dg[lo:hi], out[lo:hi], 5,
                              seed=6, first_element=first + lo, **HP)
    check(d + [out], want, "two calls")


@pytest.mark.parametrize("second", [False, True])
@pytest.mark.parametrize("n,off", [(1, 0), (127, 0), (129, 1), (100_003, 0), (100_003, 3)])
def test_conversions_match_oracle(zm, n, off, second):
    rng = np.random.default_rng(n + off)
    size = np.repeat(np.exp(rng.standard_normal(state8.n_blocks(n)) * 20), 128)[:n]
    x = (rng.standard_normal(n) * np.exp(rng.standard_normal(n) * 3) * size).astype(np.float32)
    if n > 1000:
        x[:128], x[130], x[300], x[400] = 0, np.inf, np.nan, -np.inf
        x[512:640] = rng.integers(1, 1 << 23, 128).astype(np.uint32).view(np.float32)      # subnormal
        x[640:768] = np.float32(3e38) * rng.random(128).astype(np.float32)
        x[768] = np.float32(-0.0)
        for k, (e, b) in enumerate(((7, 0x3F8), (7, 0x3F9), (-6, 0x3F8))):                 # ties
            x[1024 + k * 128:1152 + k * 128] = np.ldexp(np.float32(1 + 1 / 16), np.arange(128) % 16 - 8 + e)
    if second:
        x = np.abs(x)
    dx = torch.cat([torch.zeros(off, device=dev()), to_dev_f32(x)])[off:]
    codes, scales = u8(np.full(n, 9), off), u8(np.full(state8.n_blocks(n) + 1, 9))
    zm.zero_state8_quantize(dx, codes, scales[:-1], second_moment=second)
    wc, ws = state8.encode(x, second)
    assert_bits_equal(codes.cpu().numpy(), wc, "codes")
    assert_bits_equal(scales.cpu().numpy(), np.append(ws, 9), "scales")
    out = torch.full((n + off + 1,), 5.0, device=dev())
    zm.zero_state8_dequantize(codes, scales[:-1], out[off:off + n])
    want = state8.decode(wc, ws)
    got = host_f32(out)
    assert (got[:off] == 5).all() and got[-1] == 5
    assert np.array_equal(got[off:off + n], want, equal_nan=True)


def test_dequantize_every_code_and_scale(zm):
    codes = np.tile(np.arange(256, dtype=np.uint8), 256)
    scales = np.repeat(np.arange(256, dtype=np.uint8), 2)
    out = torch.zeros(len(codes), device=dev())
    zm.zero_state8_dequantize(u8(codes), u8(scales), out)
    got, want = host_f32(out), state8.decode(codes, scales)
    nan = np.isnan(want)
    assert (np.isnan(got) == nan).all()
    assert_bits_equal(got.view(np.uint32)[~nan], want.view(np.uint32)[~nan], "values")


def test_empty_calls_enqueue_nothing(zm):
    e, b, h = (torch.zeros(0, dtype=t, device=dev()) for t in (torch.float32, torch.uint8, torch.int16))
    zm.zero_shard_adamw8_step(e, b, b, b, b, h, h, 1, **HP)
    zm.zero_state8_quantize(e, b, b)
    zm.zero_state8_dequantize(b, b, e)
    torch.cuda.synchronize()


def test_captured_steps_replay_successive_steps(zm):
    """A graph of the scheduled flat step and the advance, and one of the table and the one-pass reduce, replayed
    seven times with new gradients between; the fourth coefficient is NaN: nothing changes and it is not counted."""
    n = 50_003
    state = make_state(n, 50)
    plan = zm.zero_partition_plan([n], 1, 1)
    forms = {}
    for form in ("flat", "table", "reduce"):
        d, out = to_dev(state), torch.zeros(n, dtype=torch.int16, device=dev())
        dg = torch.zeros(n, dtype=torch.int16, device=dev())
        clip = torch.ones(1, device=dev())
        sched = zm.AdamWSchedule(HP["lr"], HP["beta1"], HP["beta2"], HP["eps"], HP["weight_decay"])
        table = zm.MultiTensor8Table(*[[x] for x in d], [dg], [out]) if form == "table" else None
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            if form == "flat":
                zm.zero_shard_adamw8_step_scheduled(*d, dg, out, sched, seed=21, clip_scale=clip)
            elif form == "table":
                table.step_scheduled(sched, seed=21, clip_scale=clip)
            else:
                zm.zero_reduce_adamw8_step_scheduled(plan, 0, [dg], 0, n, *d, out, sched, seed=21, clip_scale=clip)
            sched.advance(clip_scale=clip)
        forms[form] = (d, out, dg, clip, sched, graph, table)
    bits, t = np.zeros(n, np.uint16), 0
    for k, coef in enumerate([1.0, 0.5, 0.75, float("nan"), 1.0, 0.25, 1.0]):
        g = make_grad(n, 60 + k)
        if math.isfinite(coef):
            t += 1
            *state, bits = oracle.adamw8_step(*state, g, t, seed=21, clip=coef, **HP)
        for form, (d, out, dg, clip, sched, graph, _) in forms.items():
            note(f"replay {k} of {form}, coefficient {coef}")
            dg.copy_(to_dev_u16(g))
            clip.fill_(coef)
            torch.cuda.synchronize()
            graph.replay()
            torch.cuda.synchronize()
            check(d + [out], list(state) + [bits], f"replay {k} {form}")
            assert sched.applied() == t


def test_steps_on_two_streams_at_once(zm):
    """Two shards on two streams, 20 steps each, interleaved, with no wait between: each as on its own."""
    n = 300_001
    states = [make_state(n, 70), make_state(n, 71)]
    ds, outs = [to_dev(s) for s in states], [torch.zeros(n, dtype=torch.int16, device=dev()) for _ in range(2)]
    g = [make_grad(n, 72), make_grad(n, 73)]
    dg = [to_dev_u16(x) for x in g]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for t in range(1, 21):
        for k in range(2):
            zm.zero_shard_adamw8_step(*ds[k], dg[k], outs[k], t, seed=k, stream=streams[k].cuda_stream, **HP)
    torch.cuda.synchronize()
    for k in range(2):
        want = states[k] + [None]
        for t in range(1, 21):
            want = oracle.adamw8_step(*want[:5], g[k], t, seed=k, **HP)
        check(ds[k] + [outs[k]], want, f"stream {k}")


@pytest.mark.parametrize("form", ["flat", "flat-device-step", "per-param", "per-param-device-step", "one-pass",
                                  "one-pass-device-step"])
def test_rank_step_with_8_bit_moments(zm, form):
    """RankStep(state_bits=8) over three steps with the operators as a step uses them, against the oracle: the
    reduce, the clip coefficient (read back), the update of the rank's part, the gather."""
    from zero_partitioned_mixed_partition_amd.step import Hyper, RankStep
    numels, n_ranks, rank, R = [1000, 37, 4096, 3, 777], 4, 2, 3
    plan = zm.zero_partition_plan(numels, n_ranks, 128)
    ref = oracle.partition_plan(numels, n_ranks, 128)
    P, S, phi = ref.padded_numel, ref.shard_numel, ref.numel
    per_param, device_step, fused = "per-param" in form, "device-step" in form, "one-pass" in form
    rs = RankStep(plan, rank, 1, Hyper(), 0.0 if fused else 1.0, dev(), device_step=device_step, per_param=per_param,
                  state_bits=8, seed=31)
    segs = ref.segments(rank)
    cuts = [(so, so + ln) for (_, _, so, ln) in segs] if per_param else [(0, S)]
    rng = np.random.default_rng(80)
    master = rng.standard_normal(S).astype(np.float32)
    m0, v0 = (rng.standard_normal(S) * 1e-3).astype(np.float32), (rng.random(S) * 1e-6).astype(np.float32)
    if per_param:
        for x, (a, b) in zip(rs.master_tensors, cuts):
            x.copy_(torch.from_numpy(master[a:b]))
        rs.load_moments([to_dev_f32(m0[a:b]) for a, b in cuts], [to_dev_f32(v0[a:b]) for a, b in cuts])
    else:
        rs.master.copy_(torch.from_numpy(master))
        rs.load_moments(to_dev_f32(m0), to_dev_f32(v0))
    parts, firsts, first = [], [], rs.first_element
    for a, b in cuts:
        m, ms = state8.encode(m0[a:b], False)
        v, vs = state8.encode(v0[a:b], True)
        parts.append([master[a:b], m, ms, v, vs])
        firsts.append(first)
        first += -(-(b - a) // 128) * 128
    rs.set_remote_partials([0.2, 0.1, 0.0, 0.05])
    reps = [torch.zeros(P, dtype=torch.int16, device=dev()) for _ in range(R)]
    for t in (1, 2, 3):
        full = [synth.normal_bf16(P, 94, synth.KIND_REPLICA, t, k, 0, phi, 0.05) for k in range(R)]
        for x, h in zip(reps, full):
            x.copy_(to_dev_u16(h))
        rs.step([(0, P, reps)])
        torch.cuda.synchronize()
        g = np.zeros(S, np.uint16)
        oracle.reduce_shard(ref, rank, full, 0, g)
        clip = 1.0 if fused else float(rs.scale.item())
        bits = host_u16(rs.param_shards[rank])
        for k, (a, b) in enumerate(cuts):
            want = oracle.adamw8_step(*parts[k], g[a:b], t, seed=31, first_element=firsts[k], clip=clip, **HP)
            if per_param:
                got = [rs.master_tensors[k], rs.exp_avg_tensors[k], rs.exp_avg_scale_tensors[k],
                       rs.exp_avg_sq_tensors[k], rs.exp_avg_sq_scale_tensors[k]]
            else:
                got = [rs.master, rs.exp_avg, rs.exp_avg_scale, rs.exp_avg_sq, rs.exp_avg_sq_scale]
            check(got + [rs.param_shards[rank][a:b]], want, f"{form} step {t} part {k}")
            parts[k] = list(want[:5])
        for (ti, toff, so, ln) in segs:
            assert_bits_equal(host_u16(rs.tensors[ti])[toff:toff + ln], bits[so:so + ln], "gathered parameters")
    assert rs.steps_applied() == 3
    m, v = rs.moments()
    for k, (a, b) in enumerate(cuts):
        for got, codes, scales in ((m[k] if per_param else m, parts[k][1], parts[k][2]),
                                   (v[k] if per_param else v, parts[k][3], parts[k][4])):
            assert_bits_equal(host_f32(got), state8.decode(codes, scales), "moments")


def test_captured_rank_step(zm):
    """A whole RankStep(state_bits=8, device_step=True) (reduce, clip, update, advance, gather) captured after one
    eager step and replayed three times with new replicas, against a second RankStep run eagerly."""
    from zero_partitioned_mixed_partition_amd.step import Hyper, RankStep
    numels, n_ranks, rank, R = [1000, 37, 4096, 3, 777], 4, 1, 2
    plan = zm.zero_partition_plan(numels, n_ranks, 128)
    P, phi = plan.padded_numel, plan.numel
    both = [RankStep(plan, rank, 1, Hyper(), 1.0, dev(), device_step=True, state_bits=8, seed=3) for _ in range(2)]
    reps = [torch.zeros(P, dtype=torch.int16, device=dev()) for _ in range(R)]
    for rs in both:
        rs.master.copy_(torch.randn(plan.shard_numel, generator=torch.Generator().manual_seed(1)))
        rs.set_remote_partials([0.2, 0.0, 0.1, 0.3])
    s = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    for t in range(1, 6):
        for k, x in enumerate(reps):
            x.copy_(to_dev_u16(synth.normal_bf16(P, 95, synth.KIND_REPLICA, t, k, 0, phi, 0.05)))
        torch.cuda.synchronize()
        both[0].step([(0, P, reps)])
        if t == 1:
            both[1].step([(0, P, reps)], stream=s.cuda_stream)
            torch.cuda.synchronize()
            with torch.cuda.graph(graph, stream=s):
                both[1].step([(0, P, reps)], stream=s.cuda_stream)
        else:
            graph.replay()
        torch.cuda.synchronize()
        for name in ("master", "exp_avg", "exp_avg_scale", "exp_avg_sq", "exp_avg_sq_scale"):
            assert torch.equal(getattr(both[0], name), getattr(both[1], name)), (t, name)
        for x, y in zip(both[0].tensors, both[1].tensors):
            assert torch.equal(x, y)
    assert both[1].steps_applied() == 5


@pytest.mark.parametrize("cut", [4096 - 64, 4096, 4096 + 128])
def test_rank_step_windows_give_the_whole_steps_bits(zm, cut):
    """Two bucket windows that meet inside the rank's shard, between blocks (one pass per window) and inside a
    block (the two calls), against one window over the whole buffer."""
    from zero_partitioned_mixed_partition_amd.step import Hyper, RankStep
    plan = zm.zero_partition_plan([9000], 2, 128)                # S = 4608, rank 0
    P, S = plan.padded_numel, plan.shard_numel
    reps = [to_dev_u16(make_grad(P, 90 + k)) for k in range(2)]
    state = make_state(S, 92)
    results = []
    for windows in ([(0, P, reps)], [(cut, P - cut, [r[cut:] for r in reps]), (0, cut, [r[:cut] for r in reps])]):
        rs = RankStep(plan, 0, len(windows), Hyper(), 0.0, dev(), state_bits=8, seed=5)
        assert rs._whole_blocks(windows) == (len(windows) == 1 or cut % 128 == 0)
        for d, h in zip((rs.master, rs.exp_avg, rs.exp_avg_scale, rs.exp_avg_sq, rs.exp_avg_sq_scale), state):
            d.copy_(torch.from_numpy(h))
        for _ in range(2):
            rs.step(windows)
        torch.cuda.synchronize()
        results.append([rs.master, rs.exp_avg, rs.exp_avg_scale, rs.exp_avg_sq, rs.exp_avg_sq_scale] + rs.tensors)
    for x, y in zip(*results):
        assert torch.equal(x, y)
