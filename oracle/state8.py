"""AdamW with its two moments held in 8 bits, and their conversions.

[ZF] "Static Memory Allocation": the fp32 moments m_t and v_t are 8 of a
parameter's 16 bytes. The 8-bit form is not on the pages. Reading taken: blocks
of 128 consecutive elements with one power-of-two scale byte b each, and an
OCP e4m3 code per element; value = e4m3(code) * 2^(b - 127), b = 255 for a
block that held an infinity or NaN (its codes are 0, it reads as NaN).

The step decodes the moments, applies adamw_step's fp32 operations to them, and
encodes the new m and v by stochastic rounding with words that depend on
(seed, step, element) only. Written from the format's definition: a code is
found by its value (sign, exponent, mantissa as integers), the rounding by a
comparison of the dropped fraction with the random draw.
"""
import numpy as np

from .adamw import adamw_step

BLOCK = 128
WINDOW = 1 << 28
_WIDE = (1 << 64) - 1


def e4m3_value(code: int) -> float:
    """OCP 8-bit float e4m3: bias 7, subnormals, 0x7F and 0xFF NaN, no infinity."""
    sign = -1.0 if code & 0x80 else 1.0
    e, f = (code >> 3) & 15, code & 7
    if e == 15 and f == 7:
        return float("nan")
    return sign * (f * 2.0 ** -9 if e == 0 else (8 + f) * 2.0 ** (e - 10))


E4M3 = np.array([e4m3_value(c) for c in range(256)])


def n_blocks(n: int) -> int:
    return -(-n // BLOCK)


def _rows(a: np.ndarray) -> np.ndarray:
    a = np.asarray(a)
    out = np.zeros(n_blocks(a.size) * BLOCK, a.dtype)
    out[:a.size] = a
    return out.reshape(-1, BLOCK)


def decode(codes: np.ndarray, scales: np.ndarray) -> np.ndarray:
    """fp32 values (float64 products, rounded once)."""
    rows = _rows(np.asarray(codes, np.uint8))
    with np.errstate(under="ignore", over="ignore"):
        out = np.ldexp(E4M3[rows], np.asarray(scales, np.int64)[:, None] - 127).astype(np.float32)
    out[np.asarray(scales) == 255] = np.nan
    return out.reshape(-1)[:len(codes)]


def words(n: int, first: int, seed: int, step: int, window: int = 0) -> np.ndarray:
    """The 32-bit random words of elements first .. first + n - 1 of one window's stream."""
    z = (seed + step * 0x6A09E667F3BCC909 + window * 0xA54FF53A5F1D36F1) & _WIDE
    z = ((z ^ (z >> 32)) * 0xBB67AE8584CAA73B) & _WIDE
    z = ((z ^ (z >> 29)) * 0x3C6EF372FE94F82B) & _WIDE
    z ^= z >> 32
    e = np.arange(first, first + n, dtype=np.uint64)
    u = np.uint64
    low = u(0xFFFFFFFF)
    q, j = e >> u(3), e & u(7)
    a = (((q & low) ^ u(z & 0xFFFFFFFF)) * u(0xA54FF53B)) & low
    a ^= a >> u(16)
    a = (((a + (q >> u(32)) + u(z >> 32)) & low) * u(0x510E527F)) & low
    a ^= a >> u(15)
    b = (a * u(0x9B05688D)) & low
    b = (b ^ (b >> u(16))) | u(1)
    return ((a + j * b) & low).astype(np.uint32)


def element_words(n: int, first: int, seed: int, step: int) -> np.ndarray:
    """The random words of elements first .. first + n - 1 of a step: each window of 2^28 elements has a
    stream of its own, numbered from the window's start."""
    parts, end = [], first + n
    while first < end:
        window, at = divmod(first, WINDOW)
        count = min(end - first, WINDOW - at)
        parts.append(words(count, at, seed, step, window) if window else words(count, at, seed, step))
        first += count
    return np.concatenate(parts) if parts else np.zeros(0, np.uint32)


def encode(x: np.ndarray, second: bool, draw: np.ndarray = None):
    """(codes, scales) of fp32 x. draw: a 20-bit integer per element (stochastic
    rounding: up where the dropped 20 bits and the draw carry), or None (to the
    nearest code, ties to even)."""
    n = len(x)
    rows = _rows(np.asarray(x, np.float32))
    big = np.abs(rows).max(axis=1)                       # NaN where the row has one
    field = (big.view(np.uint32) >> 23).astype(np.int64) & 255
    scales = np.where(field == 255, 255, np.maximum(field - 7, 0))
    finite = np.where((scales == 255)[:, None], np.float32(0), rows)
    # |x| in units of 2^-149 beside a scale of 2^-120: subnormal (below 2^23) a count of
    # them, its fraction dropped; normal the fp32 bits of the scaled value, exact.
    y = np.ldexp(np.abs(finite).astype(np.float64), 7 - scales[:, None])
    small = y < 2.0 ** -126
    bits = np.where(small, np.floor(np.ldexp(np.where(small, y, 0), 149)).astype(np.int64),
                    np.where(small, 0, y).astype(np.float32).view(np.uint32).astype(np.int64))
    kept, dropped = bits >> 20, bits & 0xFFFFF
    if draw is None:
        step = np.ldexp(1.0, np.maximum((bits >> 23), 1) - 127 - 3)      # between codes at y
        kept = np.rint(y / step).astype(np.int64)                        # exact quotient, ties to even
        kept = np.where(bits >> 23 > 0, kept + ((bits >> 23) - 1) * 8, kept)
        code = kept
    else:
        code = kept + (dropped + _rows(np.asarray(draw, np.int64)) >= 1 << 20)
    if second:
        code = np.where((code == 0) & (rows > 0), 1, code)
    code = code | (np.signbit(rows).astype(np.int64) << 7)
    code[scales == 255] = 0
    return code.reshape(-1)[:n].astype(np.uint8), scales.astype(np.uint8)


def adamw8_step(master, exp_avg, exp_avg_scale, exp_avg_sq, exp_avg_sq_scale, grad_bits, step, lr, beta1,
                beta2, eps, weight_decay, seed=0, first_element=0, clip=1.0):
    """(master, exp_avg, exp_avg_scale, exp_avg_sq, exp_avg_sq_scale, param_bits) as new arrays; param_bits
    is None when the update is skipped (non-finite clip coefficient)."""
    n = len(master)
    if not np.isfinite(np.float32(clip)):
        return tuple(np.array(a) for a in (master, exp_avg, exp_avg_scale, exp_avg_sq, exp_avg_sq_scale)) + (None,)
    with np.errstate(invalid="ignore", over="ignore", divide="ignore", under="ignore"):
        p, m, v, bits = adamw_step(master, decode(exp_avg, exp_avg_scale), decode(exp_avg_sq, exp_avg_sq_scale),
                                   grad_bits, step, lr, beta1, beta2, eps, weight_decay, clip)
    w = element_words(n, first_element, seed, step)
    mc, ms = encode(m, False, w >> np.uint32(12))
    vc, vs = encode(v, True, w & np.uint32(0xFFFFF))
    return p, mc, ms, vc, vs, bits
