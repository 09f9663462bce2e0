"""Muon on short sides whose long side is millions: the norm, which the short form takes from X X^T's fp32 sums, and the
result."""
import pytest
import torch

import oracle
from tests.gpu_util import dev, needs_gpu, note

pytestmark = [pytest.mark.gpu, needs_gpu]


@pytest.fixture(scope="module")
def zm():
    import zero_partitioned_mixed_partition_amd as m
    return m


@pytest.mark.parametrize("rows,cols", [(1, 1 << 22), (1 << 22, 1), (3, 2_000_000), (2_000_000, 3)])
@pytest.mark.parametrize("bf16", [True, False])
def test_the_norm(zm, rows, cols, bf16):
    """One step that is the identity gives X itself, each value rounded to bf16: at most half a step of bf16 off, and what the norm is off
    besides, which millions of values lie near enough to the middle of two steps to show. The values' two parts are 2^-22 off, the
    factor and the product 2^-24 each: 2^-20 in all."""
    gen = torch.Generator(device=dev()).manual_seed(1)
    x = torch.rand(rows * cols, device=dev(), generator=gen) + 1.0       # all of one sign: sums in fp32 would drift
    x = x.bfloat16() if bf16 else x
    out = torch.empty(rows * cols, dtype=torch.bfloat16, device=dev())
    zm.zero_orthogonalize(x, out, rows, cols, coefficients=[(1.0, 0.0, 0.0)], eps=0.0)
    want = x.double() / x.double().norm()
    half = torch.exp2(torch.floor(torch.log2(want)) - 8)                 # half a step
    past = float((((out.double() - want).abs() - half) / want).max())
    note(f"{rows} x {cols}: {past:.2e}")
    assert past <= 2.0 ** -20


@pytest.mark.parametrize("rows,cols", [(3, 2_000_000), (2_000_000, 3), (100, 300_000), (300_000, 70)])
def test_long_sides_against_the_formula(zm, rows, cols):
    gen = torch.Generator(device=dev()).manual_seed(2)
    x = torch.randn(rows * cols, device=dev(), generator=gen) + 0.5
    out = torch.empty(rows * cols, dtype=torch.bfloat16, device=dev())
    zm.zero_orthogonalize(x, out, rows, cols)
    m = x.view(rows, cols).double()
    m = m.T.contiguous() if rows > cols else m
    gram = m @ m.T.contiguous()
    norm = gram.diagonal().sum().sqrt()
    gram = gram / (norm + 1e-7) ** 2
    q = torch.eye(len(gram), dtype=torch.float64, device=dev())
    for a, b, c in oracle.muon.COEFFICIENTS:
        step = a * torch.eye(len(gram), dtype=torch.float64, device=dev()) + b * gram + c * (gram @ gram)
        q = step @ q
        gram = step @ gram @ step
    want = (q / (norm + 1e-7)) @ m
    got = out.view(rows, cols).double()
    got = got.T if rows > cols else got
    # at most half a step of bf16 off, and the short form's 3e-5 of the result's root mean square
    half = torch.exp2(torch.floor(torch.log2(want.abs().clamp_min(1e-30))) - 8)
    rms = want.square().mean().sqrt()
    past = float((((got - want).abs() - half) / rms).max())
    note(f"{rows} x {cols}: {past:.2e}")
    assert past <= 8 * 3e-5
