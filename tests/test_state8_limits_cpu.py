"""The element limit of the 8-bit entry points: 2^48 and one more, exactly, before any HIP call (the addresses are
never dereferenced; at the limit the arrays overlap, so nothing is enqueued)."""
import ctypes

import pytest

HP = (1e-3, 0.9, 0.999, 1e-8, 0.01)
LIMIT = 1 << 48


@pytest.fixture(scope="module")
def zm():
    import zero_partitioned_mixed_partition_amd as m
    return m


def _calls(zm, n):
    b = zm._binding
    a = [ctypes.c_void_p(0x1000000 * (k + 1)) for k in range(7)]
    plan = zm.zero_partition_plan([n], 1, 1)
    reps = (ctypes.c_void_p * 1)(0x100000000)
    return {
        "step": lambda: b._adamw8(*a, n, 128, 1, *HP, 0, None, None),
        "reduce": lambda: b._reduce_adamw8(plan.handle, 0, reps, 1, 0, n, *a[:5], a[6], None, 0, 1, *HP, 0, None, None),
        "quantize": lambda: b._quantize8(a[0], n, 0, a[1], a[2], None),
        "dequantize": lambda: b._dequantize8(a[1], a[2], n, a[0], None),
    }


@pytest.mark.parametrize("form", ["step", "reduce", "quantize", "dequantize"])
def test_the_limit_is_2_48_elements(zm, form):
    E, R = zm._binding.ZERO_EINVAL, zm._binding.ZERO_ERANGE
    for n in (LIMIT + 1, 2 * LIMIT, 1 << 52):
        assert _calls(zm, n)[form]() == R, n
        assert "2^48" in zm.zero_last_error()
    assert _calls(zm, LIMIT)[form]() == E and "overlaps" in zm.zero_last_error()


def test_lengths_whose_bytes_pass_64_bits(zm):
    """4 n bytes do not fit 64 bits: refused by the limit, not by a wrapped range."""
    b, R = zm._binding, zm._binding.ZERO_ERANGE
    a = [ctypes.c_void_p(0x1000000 * (k + 1)) for k in range(7)]
    for n in (1 << 62, (1 << 63) - 1):
        assert b._adamw8(*a, n, 0, 1, *HP, 0, None, None) == R
        assert b._quantize8(a[0], n, 0, a[1], a[2], None) == R
        assert b._dequantize8(a[1], a[2], n, a[0], None) == R
