"""Muon's precision on matrices that are hard for it, with short sides past 128: few strong directions over a floor, low rank,
falling singular values, and many steps. Against the oracle's formula in float64 on the GPU.

Bounds. Every held value is rounded to fp16, 2^-11 / sqrt(3) = 2.8e-4 of its norm, and each step multiplies what lies in a
direction that X hardly has by its a = 3.4445. X's own roundings are carried along. Those of A, C and Q (of a pair of steps T, A'
and the second C too) reach such directions only from the strong ones, r of m, whose share of a rounding is sqrt(r / m), at most
0.7: 2.0e-4 each of the strong directions' norm, which is at most the result's. While the strong values are still below 1/2 (the
first two steps, of up to 32 of them) what A adds to C is below that of a I, and little is left of these roundings; the three
products of the third step, or six of a second pair, are multiplied by 3.4445^2 = 11.9: 2.0e-4 sqrt(6) 11.9 = 5.8e-3. (Without X's
roundings carried along those of X after the first pair, 2.8e-4, are multiplied by 3.4445^3 = 41: 1.2e-2.) With the rounding to bf16
(2.3e-3) in quadrature and a tenth more FIVE = 7e-3. Each step more multiplies by 3.4445: four more, of matrices whose values lie
above 1e-3 of the largest and so reach 0.4 by themselves in seven steps, leave two for roundings to grow in, 5.8e-3 11.9 = 0.07 at
most, NINE = 6e-2.
"""
import numpy as np
import pytest
import torch

import oracle
from tests.gpu_util import dev, needs_gpu, note

pytestmark = [pytest.mark.gpu, needs_gpu]

FIVE, NINE = 7e-3, 6e-2
USUAL = oracle.muon.COEFFICIENTS


@pytest.fixture(scope="module")
def zm():
    import zero_partitioned_mixed_partition_amd as m
    return m


def in_64_bits(x, steps, eps=1e-7):
    if x.shape[0] > x.shape[1]:
        return in_64_bits(x.T.contiguous(), steps, eps).T
    x = x.double()
    x = x / (x.norm() + eps)
    for a, b, c in steps:
        gram = x @ x.T.contiguous()
        x = a * x + (b * gram + c * (gram @ gram)) @ x
    return x


def spectrum(kind, m):
    k = np.arange(m)
    return {"rank 1": (k < 1) * 1.0, "rank 3": (k < 3) * 1.0, "32 over 1e-3": np.where(k < 32, 1.0, 1e-3),
            "8 over 1e-4": np.where(k < 8, 1.0, 1e-4), "half over 1e-3": np.where(k < m // 2, 1.0, 1e-3),
            "half over 1e-2": np.where(k < m // 2, 1.0, 1e-2), "1/k": 1.0 / (1 + k), "1/k^2": (1.0 + k) ** -2.0,
            "1e-3 by ratios": 10.0 ** (-3 * k / m), "1e-6 by ratios": 10.0 ** (-6 * k / m), "flat": np.ones(m)}[kind]


def matrix(kind, rows, cols, seed=0):
    """float64 on the GPU with these singular values and random directions."""
    gen = torch.Generator(device=dev()).manual_seed(seed)
    m = min(rows, cols)
    u = torch.linalg.qr(torch.randn(rows, m, device=dev(), dtype=torch.float64, generator=gen))[0]
    v = torch.linalg.qr(torch.randn(cols, m, device=dev(), dtype=torch.float64, generator=gen))[0]
    return (u * torch.from_numpy(spectrum(kind, m)).to(dev())) @ v.T.contiguous()


def off(zm, x, bf16, steps):
    """The error's Frobenius norm over the result's, and the largest singular value of the error."""
    rows, cols = x.shape
    x = x.bfloat16() if bf16 else x.float()
    out = torch.empty(x.numel(), dtype=torch.bfloat16, device=dev())
    zm.zero_orthogonalize(x.reshape(-1), out, rows, cols, coefficients=steps)
    want = in_64_bits(x, steps)
    d = out.view(rows, cols).double() - want
    return float(d.norm() / want.norm()), float(torch.linalg.matrix_norm(d, 2))


KINDS = ["rank 1", "rank 3", "32 over 1e-3", "8 over 1e-4", "half over 1e-3", "half over 1e-2", "1/k", "1/k^2", "1e-3 by ratios",
         "1e-6 by ratios", "flat"]


@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("shape", [(200, 260), (260, 200), (384, 768), (768, 768), (300, 1500)])
@pytest.mark.parametrize("kind", KINDS)
def test_five_steps(zm, kind, shape, bf16):
    # rounding to bf16 gives a matrix of few directions a floor of its own, 2.3e-3 of it, that the steps then raise: part of the input
    error, largest = off(zm, matrix(kind, *shape), bf16, USUAL)
    note(f"{kind} {shape} bf16={bf16}: {error:.2e}, largest {largest:.2e}")
    assert error <= FIVE


@pytest.mark.parametrize("shape", [(300, 500), (500, 300), (768, 800)])
@pytest.mark.parametrize("kind", ["32 over 1e-3", "half over 1e-3", "half over 1e-2", "1/k", "1e-3 by ratios", "flat"])
def test_nine_steps(zm, kind, shape):
    error, largest = off(zm, matrix(kind, *shape), False, USUAL[:1] * 9)
    note(f"{kind} {shape}: {error:.2e}, largest {largest:.2e}")
    assert error <= NINE


@pytest.mark.parametrize("rows,cols", [(4096, 4096), (1024, 4096), (4100, 1100)])
def test_large_ones(zm, rows, cols):
    """32 directions over 1e-3 of them: tiles of 256, and two pairs of steps where one side is much the longer."""
    gen = torch.Generator(device=dev()).manual_seed(3)
    normal = lambda *s: torch.randn(*s, device=dev(), generator=gen, dtype=torch.float64)  # noqa: E731
    x = normal(rows, 32) @ normal(32, cols)
    x += 1e-3 * torch.linalg.matrix_norm(x, 2) / (rows ** 0.5 + cols ** 0.5) * normal(rows, cols)
    error, largest = off(zm, x, False, USUAL)
    note(f"{rows} x {cols}: {error:.2e}, largest {largest:.2e}")
    assert error <= FIVE
