"""The 8-bit-moment oracle against definitions outside it: torch's e4m3 and e8m0
conversions, closed forms of the rounding, and a pure-Python count of the random
words."""
import numpy as np
import pytest
import torch

import oracle
from oracle import state8


def _torch_value(codes, scales):
    c = torch.from_numpy(codes).view(torch.float8_e4m3fn).double()
    s = torch.from_numpy(np.repeat(scales, state8.BLOCK)[:len(codes)]).view(torch.float8_e8m0fnu).double()
    return (c * s).float().numpy()


def test_decode_matches_torch_for_every_code_and_scale():
    for scale in range(256):
        codes = np.arange(256, dtype=np.uint8)
        scales = np.full(2, scale, np.uint8)
        got, want = state8.decode(codes, scales), _torch_value(codes, scales)
        assert np.array_equal(got, want, equal_nan=True), scale


@pytest.mark.parametrize("power", [-130, -40, -9, 0, 5, 100])
def test_nearest_codes_match_torchs_conversion(power):
    rng = np.random.default_rng(1)
    x = np.ldexp(rng.standard_normal(128 * 64) * np.exp(rng.standard_normal(128 * 64) * 4), power).astype(np.float32)
    codes, scales = state8.encode(x, False)
    units = np.ldexp(x.astype(np.float64), 127 - np.repeat(scales, 128).astype(np.int64)).astype(np.float32)
    assert np.abs(units).max() < 256 and (power < -110 or np.abs(units).max() >= 128)
    want = torch.from_numpy(units).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(codes, want)
    # half a step of 2^-3 relative, or half the least step
    err = np.abs(state8.decode(codes, scales).astype(np.float64) - x)
    step = np.maximum(np.abs(x) / 16, np.ldexp(0.5, np.repeat(scales, 128).astype(np.int64) - 127 - 9))
    assert (err <= step * (1 + 1e-6)).all()


def test_codes_survive_a_round_trip():
    rng = np.random.default_rng(2)
    codes = rng.integers(0, 0x78, (40, 128)).astype(np.uint8)      # below 2^8
    codes[:, 0] = 0x75                                             # each block's maximum in [2^7, 2^8)
    codes |= (rng.integers(0, 2, codes.shape) << 7).astype(np.uint8)
    scales = rng.integers(1, 240, 40).astype(np.uint8)
    flat = codes.reshape(-1)
    again, s2 = state8.encode(state8.decode(flat, scales), False)
    assert np.array_equal(again, flat) and np.array_equal(s2, scales)


@pytest.mark.parametrize("value", [1.0, 1.03, 1.99, 0.37, 3.3e-3, 9e-6])
def test_stochastic_rounding_is_unbiased_over_all_draws(value):
    """All 2^20 draws once: the mean of the rounded values is the value itself,
    exactly where y is a normal number, else to y's own rounding (2^-20 of the
    least code)."""
    rows = np.full((1 << 14, 128), 1.5, np.float32)                 # half of each block sets the scale
    rows[:, :64] = value
    draws = np.zeros(rows.shape, np.int64)
    draws[:, :64] = np.arange(1 << 20).reshape(-1, 64)
    codes, scales = state8.encode(rows.reshape(-1), False, draws.reshape(-1))
    values = state8.decode(codes, scales).reshape(-1, 128)[:, :64].astype(np.float64)
    assert (scales == 120).all()                                    # 1.5 is 192 units of 2^-7
    assert abs(values.mean() - float(np.float32(value))) <= 2.0 ** -16 * 2.0 ** -20
    assert len(np.unique(values)) <= 2


def test_zeros_positive_minimum_and_non_finite_blocks():
    x = np.zeros(128 * 5, np.float32)
    x[128], x[129], x[130] = 1.0, 1e-30, 0.0        # far below the block's least code
    x[256], x[257] = np.inf, 1.0
    x[384] = np.nan
    x[512], x[513] = 1e-45, 1e-40                   # subnormal block
    for second in (False, True):
        codes, scales = state8.encode(x, second, np.zeros(len(x), np.int64))
        assert (codes[:128] == 0).all() and scales[0] == 0
        assert codes[129] == (1 if second else 0) and codes[130] == 0
        assert scales[2] == 255 and scales[3] == 255 and (codes[256:512] == 0).all()
        back = state8.decode(codes, scales)
        assert np.isnan(back[256:512]).all() and back[128] == 1.0
        assert scales[4] == 0 and np.isfinite(back[512:]).all()


def test_words_match_a_pure_python_count():
    m32, m64 = (1 << 32) - 1, (1 << 64) - 1
    for seed, step, first in [(0, 1, 0), (12345678901234567890, 7, 128), (3, 1 << 40, (1 << 36) - 128)]:
        z = (seed + step * 0x6A09E667F3BCC909) & m64
        z = ((z ^ z >> 32) * 0xBB67AE8584CAA73B) & m64
        z = ((z ^ z >> 29) * 0x3C6EF372FE94F82B) & m64
        z ^= z >> 32
        got = state8.words(300, first, seed, step)
        for i in range(300):
            q, j = (first + i) // 8, (first + i) % 8
            a = ((q & m32 ^ z & m32) * 0xA54FF53B) & m32
            a ^= a >> 16
            a = ((a + (q >> 32) + (z >> 32)) * 0x510E527F) & m32
            a ^= a >> 15
            b = a * 0x9B05688D & m32
            b = (b ^ b >> 16) | 1
            assert int(got[i]) == (a + j * b) & m32


@pytest.mark.parametrize("p", [0.008, 0.3])
def test_words_are_uniform_and_uncorrelated(p):
    """Rates of the event draw >= 1 - p, in both draws of an element, in pairs of
    neighbours and of successive steps: within 5 standard deviations."""
    n = 1 << 18
    cut = (1 - p) * 2 ** 20
    hits = []
    for step in (1, 2):
        w = state8.words(n, 0, 99, step)
        hits.append((w >> 12 >= cut, (w & 0xFFFFF) >= cut))
    q = round(p * 2 ** 20) / 2 ** 20
    for h in hits[0] + hits[1]:
        assert abs(h.mean() - q) < 5 * np.sqrt(q / n)
    pairs = [(hits[0][0], hits[0][1]), (hits[0][0], hits[1][0]), (hits[0][1], hits[1][1])]
    for lag in (1, 2, 4, 8, 128):
        pairs += [(hits[0][0][lag:], hits[0][0][:-lag]), (hits[0][1][lag:], hits[0][1][:-lag])]
    for a, b in pairs:
        assert abs((a & b).mean() - q * q) < 5 * np.sqrt(q * q / n * (1 + 4 * q))


def test_a_slow_second_moment_keeps_its_mean():
    """v starts at 4 g^2 with g constant. After 500 steps the fp32 recursion gives
    g^2 (1 + 3 * 0.999^500) = 2.819 g^2. Each rounding adds a variance of at most
    drift * step <= (0.003 g^2)(0.5 g^2), 0.75 g^4 in all, so the mean over 32,768
    elements has a standard deviation below 0.0048 g^2; 0.024 is five of them.
    Rounding to nearest leaves every code where it was: 4 g^2."""
    n, g = 32768, 2.0 ** -10
    hp = dict(lr=1e-3, beta1=0.9, beta2=0.999, eps=1e-8, weight_decay=0.0)
    grad = oracle.f32_to_bf16(np.full(n, g, np.float32))
    zeros, zs = np.zeros(n, np.uint8), np.zeros(state8.n_blocks(n), np.uint8)
    v, vs = state8.encode(np.full(n, 4 * g * g, np.float32), True)
    p, m, ms = np.zeros(n, np.float32), zeros, zs
    for t in range(1, 501):
        p, m, ms, v, vs, _ = oracle.adamw8_step(p, m, ms, v, vs, grad, t, seed=5, **hp)
    want = g * g * (1 + 3 * 0.999 ** 500)
    mean = state8.decode(v, vs).astype(np.float64).mean()
    assert abs(mean - want) < 0.024 * g * g, (mean / (g * g), want / (g * g))
    w = np.float32(4 * g * g) * np.float32(0.999) + np.float32(0.001 * g * g)
    c, s = state8.encode(np.full(128, w, np.float32), True)
    assert state8.decode(c, s)[0] == 4 * g * g


def test_step_on_exact_states_equals_the_32_bit_step():
    """On zero moments the master weights and parameters are the 32-bit step's, and the moments its
    rounded to a neighbouring code."""
    rng = np.random.default_rng(4)
    n = 1000
    p = rng.standard_normal(n).astype(np.float32)
    g = oracle.f32_to_bf16(rng.standard_normal(n).astype(np.float32) * 1e-3)
    hp = dict(lr=1e-3, beta1=0.9, beta2=0.999, eps=1e-8, weight_decay=0.01)
    z, zs = np.zeros(n, np.uint8), np.zeros(state8.n_blocks(n), np.uint8)
    got = oracle.adamw8_step(p, z, zs, z, zs, g, 1, seed=3, clip=0.5, **hp)
    want = oracle.adamw_step(p, np.zeros(n, np.float32), np.zeros(n, np.float32), g, 1, clip=0.5, **hp)
    assert np.array_equal(got[0], want[0]) and np.array_equal(got[5], want[3])
    for codes, scales, ref in ((got[1], got[2], want[1]), (got[3], got[4], want[2])):
        least = np.ldexp(1.0, np.repeat(scales, 128)[:n].astype(np.int64) - 127 - 9)
        assert (np.abs(state8.decode(codes, scales).astype(np.float64) - ref)
                <= np.maximum(np.abs(ref) / 8, least)).all()


def test_windows_round_as_the_whole():
    rng = np.random.default_rng(6)
    n = 128 * 9 + 40
    p = rng.standard_normal(n).astype(np.float32)
    g = oracle.f32_to_bf16(rng.standard_normal(n).astype(np.float32))
    m, ms = state8.encode(rng.standard_normal(n).astype(np.float32), False)
    v, vs = state8.encode(np.abs(rng.standard_normal(n)).astype(np.float32), True)
    hp = dict(lr=1e-3, beta1=0.9, beta2=0.999, eps=1e-8, weight_decay=0.01)
    whole = oracle.adamw8_step(p, m, ms, v, vs, g, 9, seed=8, first_element=1280, **hp)
    cuts = [0, 128, 640, n]
    parts = [oracle.adamw8_step(p[a:b], m[a:b], ms[a // 128:-(-b // 128)], v[a:b], vs[a // 128:-(-b // 128)], g[a:b],
                                9, seed=8, first_element=1280 + a, **hp) for a, b in zip(cuts, cuts[1:])]
    for k in range(6):
        assert np.array_equal(whole[k], np.concatenate([q[k] for q in parts])), k
