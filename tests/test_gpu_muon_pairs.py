"""Muon's steps in pairs, which sides of unlike length take, with each tile of the square products: the product that joins a
later pair is computed in full, its tiles above the diagonal by workgroups of their own. 32 directions over 1e-3 of them, against
the oracle's formula in float64 on the GPU; the bound is that of tests/test_gpu_muon_spectra.py."""
import pytest
import torch

import oracle
from tests.gpu_util import dev, needs_gpu, note
from tests.test_gpu_muon_spectra import FIVE, in_64_bits

pytestmark = [pytest.mark.gpu, needs_gpu]


@pytest.fixture(scope="module")
def zm():
    import zero_partitioned_mixed_partition_amd as m
    return m


def few_directions(rows, cols, seed):
    gen = torch.Generator(device=dev()).manual_seed(seed)
    normal = lambda *s: torch.randn(*s, device=dev(), generator=gen)  # noqa: E731
    strong = (rows ** 0.5 + 32 ** 0.5) * (cols ** 0.5 + 32 ** 0.5)          # the largest singular value, near enough
    return normal(rows, 32) @ normal(32, cols) + 1e-3 * strong / (rows ** 0.5 + cols ** 0.5) * normal(rows, cols)


@pytest.mark.parametrize("count,rows,cols", [(1, 150, 6000), (3, 6100, 155), (1, 4100, 1100), (1, 2050, 8200), (1, 3000, 12000),
                                             (1, 6000, 18001)])
@pytest.mark.parametrize("bf16", [True, False])
def test_pairs(zm, count, rows, cols, bf16):
    x = torch.stack([few_directions(rows, cols, 5 + k) for k in range(count)])
    x = x.bfloat16() if bf16 else x
    n = x.numel()
    out = [torch.full((n + 64,), 0x55, dtype=torch.int16, device=dev()) for _ in range(2)]
    for o in out:
        zm.zero_orthogonalize(x.view(-1), o[:n], rows, cols)
    assert torch.equal(out[0], out[1]) and (out[0][n:] == 0x55).all()
    got = out[0][:n].view(torch.bfloat16).view(count, rows, cols)
    for k in range(count):
        want = in_64_bits(x[k], oracle.muon.COEFFICIENTS)
        error = float((got[k].double() - want).norm() / want.norm())
        note(f"{rows} x {cols} bf16={bf16}: {error:.2e}")
        assert error <= FIVE


def test_a_list_in_pairs_is_its_matrices(zm):
    """Unlike sides, wide and tall, in one launch a product: master weights by the whole update, against 64 bits."""
    shapes = [(150, 6000), (3000, 400), (200, 2100), (64, 5000), (4100, 1100)]
    grads = [few_directions(r, c, 20 + k) * 1e-3 for k, (r, c) in enumerate(shapes)]
    masters = [torch.zeros(r * c, device=dev()) for r, c in shapes]
    momenta = [2 * g.reshape(-1) for g in grads]         # momentum 0.5 and no gradient: the matrix itself
    zeros = [torch.zeros(r * c, dtype=torch.int16, device=dev()) for r, c in shapes]
    outs = [torch.zeros_like(z) for z in zeros]
    zm.MuonTable(masters, momenta, zeros, outs, shapes, [1.0] * len(shapes)).step(lr=1.0, momentum=0.5, nesterov=False)
    for (r, c), g, p in zip(shapes, grads, masters):
        want = -in_64_bits(g, oracle.muon.COEFFICIENTS)
        error = float((p.view(r, c).double() - want).norm() / want.norm())
        note(f"{r} x {c}: {error:.2e}")
        assert error <= FIVE
