"""The least code of a positive second moment: what the stochastic rounding keeps in the mean, and what it does not."""
import numpy as np
import pytest

import oracle
from oracle import state8

LEAST = 2.0 ** -9 / 192         # the least code beside a block's largest of 1.5 (192 code units)


def _mean(value):
    """The mean decoded second moment over all 2^20 draws, beside 1.5 in the same block."""
    rows = np.full((1 << 14, 128), 1.5, np.float32)
    rows[:, :64] = value
    draws = np.zeros(rows.shape, np.int64)
    draws[:, :64] = np.arange(1 << 20).reshape(-1, 64)
    codes, scales = state8.encode(rows.reshape(-1), True, draws.reshape(-1))
    return state8.decode(codes, scales).reshape(-1, 128)[:, :64].astype(np.float64).mean()


@pytest.mark.parametrize("ratio", [1.0, 1.25, 1.9, 7.3, 100.0])
def test_the_mean_is_kept_from_the_least_code_on(ratio):
    value = np.float32(1.5 * LEAST * ratio)
    # bits of y below fp32's least subnormal are dropped: 2^-20 of the least code
    assert abs(_mean(value) - float(value)) <= 1.5 * LEAST * 2.0 ** -20


@pytest.mark.parametrize("ratio", [0.999, 0.5, 0.01, 1e-6])
def test_below_the_least_code_a_positive_value_reads_as_it(ratio):
    """2^-17 to 2^-16 of the block's largest: here 2^-9 / 192 of it. The mean is the least code, not the value."""
    assert _mean(np.float32(1.5 * LEAST * ratio)) == 1.5 * LEAST
    assert 2.0 ** -17 <= LEAST <= 2.0 ** -16


def test_a_block_of_large_and_tiny_second_moments_over_steps():
    """One element of a block has gradients of 1, the others of 2^-12 (squares 2^-24 of the largest): their v stays
    at the block's least code from the first step on, where the 32-bit v is the gradient's square in the mean, and
    their steps shrink by the root of the ratio, never below it."""
    n, steps = 1024, 60
    small = 2.0 ** -12
    g = np.full(n, small, np.float32)
    g[::128] = 1.0
    grad = oracle.f32_to_bf16(g)
    hp = dict(lr=1e-3, beta1=0.0, beta2=0.999, eps=1e-30, weight_decay=0.0)
    z, zs = np.zeros(n, np.uint8), np.zeros(state8.n_blocks(n), np.uint8)
    p8, m, ms, v, vs = np.zeros(n, np.float32), z, zs, z, zs
    for t in range(1, steps + 1):
        before = p8
        p8, m, ms, v, vs, _ = oracle.adamw8_step(p8, m, ms, v, vs, grad, t, seed=3, **hp)
        held = state8.decode(v, vs).reshape(-1, 128)[:, 1:]
        least = np.ldexp(1.0, vs.astype(np.int64) - 127 - 9)[:, None]
        assert (held == least).all() and (least > 2.0 ** -24 * (1 - 0.999 ** t)).all()
        if t > 1:
            # the step taken: lr g sqrt(bias) / sqrt(v) with v between the decayed floor and the new one
            taken = np.abs((p8 - before).reshape(-1, 128)[:, 1:]).astype(np.float64)
            v_used = 0.999 * last + 0.001 * small * small
            want = 1e-3 * small * np.sqrt(1 - 0.999 ** t) / np.sqrt(v_used)
            # p accumulates: half an ulp of |p8| <= 0.1 a step, and a few roundings of the ratio
            assert np.allclose(taken, np.broadcast_to(want, taken.shape), rtol=1e-5, atol=2.0 ** -27)
            assert (taken < 1e-3).all()
        last = least


@pytest.mark.parametrize("second", [False, True])
def test_what_a_trip_through_fp32_keeps(second):
    """Stochastically rounded moments decoded and encoded again, to nearest: blocks keep their bytes unless their
    largest was rounded up to 2^8 code units. Those get the next scale; each value moves by at most half the new
    scale's step below the normal codes (2^-10 units), and a second moment by at most the new least code."""
    rng = np.random.default_rng(2)
    n = 128 * 4000
    x = (rng.standard_normal(n) * 1e-3).astype(np.float32)
    x = x * x if second else x
    codes, scales = state8.encode(x, second, rng.integers(0, 1 << 20, n))
    values = state8.decode(codes, scales)
    again, scales2 = state8.encode(values, second)
    full = ((codes.reshape(-1, 128) & 0x7F).max(axis=1) == 0x78)            # 2^8
    assert 0 < full.sum() < len(full) // 10
    assert np.array_equal(scales2, scales + full)
    same = codes.reshape(-1, 128)[~full] & 0x7F
    assert np.array_equal(again.reshape(-1, 128)[~full] & 0x7F, same)
    moved = np.abs(state8.decode(again, scales2).astype(np.float64) - values).reshape(-1, 128)[full]
    unit = np.ldexp(1.0, scales2.astype(np.int64) - 127)[full][:, None]
    assert (moved <= unit * (2.0 ** -9 if second else 2.0 ** -10)).all()
