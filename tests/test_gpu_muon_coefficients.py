"""Muon's coefficients other than the usual five, on both sides of a short side of 128, against the 64-bit oracle.

Tolerance: that of tests/test_muon_program_cpu.py, 2e-2 of the result's norm for steps whose slope reaches 5 where the result
is near 1, with bf16's rounding (2.3e-3) below it in quadrature.
"""
import numpy as np
import pytest
import torch

import oracle
from tests.gpu_util import dev, host_u16, needs_gpu, note, to_dev_f32, to_dev_u16
from tests.test_muon_program_cpu import POLAR, SAFETY, USUAL, divided

pytestmark = [pytest.mark.gpu, needs_gpu]

NEAR = 2e-2


@pytest.fixture(scope="module")
def zm():
    import zero_partitioned_mixed_partition_amd as m
    return m


def gradients(seed, rows, cols):
    rng = np.random.default_rng(seed)
    x = rng.normal(size=(rows, cols)) + 0.5 * (rng.normal(size=(rows, 3)) * [1.0, 0.7, 0.5]) @ rng.normal(size=(3, cols))
    return (x * 1e-3).astype(np.float32)


def orthogonalized(zm, x, bf16, steps):
    if bf16:
        bits = oracle.f32_to_bf16(x)
        d, x = to_dev_u16(bits.reshape(-1)), oracle.bf16_to_f32(bits)
    else:
        d = to_dev_f32(x.reshape(-1))
    out = torch.empty(x.size, dtype=torch.int16, device=dev())
    zm.zero_orthogonalize(d, out, *x.shape, coefficients=steps)
    return oracle.bf16_to_f32(host_u16(out)).astype(np.float64).reshape(x.shape), x


@pytest.mark.parametrize("bf16", [True, False])
@pytest.mark.parametrize("shape", [(64, 200), (120, 90), (150, 260), (300, 170), (500, 520)])
@pytest.mark.parametrize("name", ["published", "over 1.003", "over 1.01, but the last", "four"])
def test_polar_express(zm, name, shape, bf16):
    """As published, where X is taken a little smaller (SAFETY) in all steps but the last, and with a safety of the caller's.
    (Four of the steps are not too steep for the two fp16 parts of short sides, which take them as they are.)"""
    note(f"{name} {shape} bf16={bf16}")
    steps = {"published": POLAR, "over 1.003": divided(POLAR, 1.003), "four": POLAR[:4],
             "over 1.01, but the last": divided(POLAR[:4], 1.01) + [POLAR[4]]}[name]
    taken = divided(steps[:-1], SAFETY) + [steps[-1]] if name == "published" or (
        name == "four" and min(shape) > 128) else steps
    got, x = orthogonalized(zm, gradients(sum(shape), *shape), bf16, steps)
    want = oracle.muon.orthogonalize(x, taken)
    assert np.linalg.norm(got - want) <= NEAR * np.linalg.norm(want), np.linalg.norm(got - want) / np.linalg.norm(want)


@pytest.mark.parametrize("shape", [(1, 300), (1, 1), (200, 1)])
def test_polar_express_of_a_vector(zm, shape):
    """Its one singular value is the norm, the edge itself, where these steps grow steeply: of X / SAFETY they do not."""
    got, x = orthogonalized(zm, gradients(1, *shape), False, POLAR)
    want = oracle.muon.orthogonalize(x, divided(POLAR[:4], SAFETY) + [POLAR[4]])
    assert np.linalg.norm(got - want) <= 0.1 * np.linalg.norm(want)


@pytest.mark.parametrize("bf16", [True, False])
@pytest.mark.parametrize("shape", [(150, 260), (260, 150), (200, 200)])
@pytest.mark.parametrize("n", [1, 2, 3, 4])
def test_a_first_step_that_is_not_paired(zm, shape, n, bf16):
    """|a| > 4 in the first step: its apply is one alone, which adds what rounding X left and is not the last product."""
    steps = [(5.023, -14.301, 10.485), USUAL, (2.0, -1.5, 0.5), (1.5, -0.5, 0.0)][:n]
    got, x = orthogonalized(zm, gradients(n, *shape), bf16, steps)
    want = oracle.muon.orthogonalize(x, steps)
    assert np.linalg.norm(got - want) <= NEAR * np.linalg.norm(want), np.linalg.norm(got - want) / np.linalg.norm(want)


@pytest.mark.parametrize("shape", [(150, 260), (260, 150), (300, 300)])
def test_other_coefficients_past_128(zm, shape):
    """Steps of their own each, growing and shrinking, and one that is the identity."""
    steps = ((2.0, -1.5, 0.5), (1.5, -0.5, 0.0), (1.0, 0.0, 0.0), (1.875, -1.25, 0.375), (0.25, 0.0, 0.0))
    for n in (1, 3, 5):
        got, x = orthogonalized(zm, gradients(n, *shape), False, steps[:n])
        want = oracle.muon.orthogonalize(x, steps[:n])
        assert np.linalg.norm(got - want) <= 5e-3 * np.linalg.norm(want), n


def test_coefficients_that_grow_are_refused(zm):
    x = to_dev_f32(gradients(1, 150, 260).reshape(-1))
    out = torch.zeros(x.numel(), dtype=torch.int16, device=dev())
    with pytest.raises(RuntimeError, match="grow past 2\\^20"):
        zm.zero_orthogonalize(x, out, 150, 260, coefficients=[(1.0, 1.0, 1.0)] * 6)
    assert not out.any()
