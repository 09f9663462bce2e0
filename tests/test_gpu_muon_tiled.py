"""The tiled form of Muon (short sides past 128) where values are extreme or not finite, and its stacks and skipped updates:
what tests/test_gpu_muon.py asks of every form at sizes that all take the short one. Tolerances are its."""
import numpy as np
import pytest
import torch

import oracle
from tests.gpu_util import dev, host_f32, host_u16, needs_gpu, note, to_dev_f32
from tests.test_gpu_muon import FROBENIUS, HYPER, LEAST, check, composed, matrices, on_device, run, same, state

pytestmark = [pytest.mark.gpu, needs_gpu]

# Wide and tall, of every tile that such calls take.
SIDES = [(140, 156), (190, 170), (190, 230), (520, 300)]


@pytest.fixture(scope="module")
def zm():
    import zero_partitioned_mixed_partition_amd as m
    return m


@pytest.mark.parametrize("size", [1e-38, 1e-30, 1e-12, 1.0, 1e12, 1e30, 1e36])
@pytest.mark.parametrize("eps", [0.0, 1e-7, 1.0])
@pytest.mark.parametrize("rows,cols", SIDES)
def test_sizes_of_values(zm, size, eps, rows, cols):
    """Any magnitude fp32 holds; eps matters where the norm is near it."""
    x = matrices(5, 1, rows, cols, 1.0, strong=0)
    x = (x.astype(np.float64) * size).astype(np.float32)
    got, x = run(zm, x, False, eps=eps)
    want = [oracle.muon.orthogonalize(m, eps=eps) for m in x]
    if np.abs(want[0]).max() < 1e-6:        # norm far below eps
        w = np.abs(want[0])
        off = np.abs(oracle.bf16_to_f32(got[0]).astype(np.float64) - want[0])
        assert (off <= 2.0 ** -8 * w + 8 * 4e-3 * np.sqrt(np.mean(w * w)) + LEAST).all()
    else:
        check(got, want, (size, eps))


@pytest.mark.parametrize("bf16", [True, False])
@pytest.mark.parametrize("rows,cols", SIDES)
def test_zeros_infinities_and_nans_stay_in_their_matrix(zm, rows, cols, bf16):
    x = matrices(6, 7, rows, cols)
    clean, _ = run(zm, x, bf16)
    x[1] = 0.0
    x[2, 3, 4] = np.inf
    x[3, rows - 1, cols - 1] = -np.inf
    x[4, 0, 0] = np.nan
    x[5] = -0.0
    for eps in (1e-7, 0.0):
        got, _ = run(zm, x, bf16, eps=eps)
        f = oracle.bf16_to_f32(got)
        assert not f[1].any() and not f[5].any()
        assert np.isnan(f[2:5]).all()
    got, _ = run(zm, x, bf16)
    assert (got[[0, 6]] == clean[[0, 6]]).all()


@pytest.mark.parametrize("rows,cols", SIDES)
def test_a_value_past_the_norm_of_the_rest(zm, rows, cols):
    """One element of 1e30 among those of 1: the rest are 1e-30 of the norm, which fp16 does not hold."""
    x = matrices(7, 1, rows, cols, 1.0)
    x[0, 5, 7] = 1e30
    got, x = run(zm, x, False)
    f = oracle.bf16_to_f32(got[0]).astype(np.float64)
    want = oracle.muon.orthogonalize(x[0])
    assert np.isfinite(f).all() and abs(f[5, 7] - want[5, 7]) <= 2e-2
    f[5, 7] = want[5, 7]
    assert np.linalg.norm(f - want, 2) < 0.02


def test_a_stack_is_its_matrices(zm):
    """Bit for bit, and the same bits twice: five of 150 x 200 and one of them take the same tiles."""
    x = matrices(9, 5, 150, 200)
    got, _ = run(zm, x, False)
    again, _ = run(zm, x, False)
    assert (got == again).all()
    for i in range(5):
        one, _ = run(zm, x[i:i + 1], False)
        assert (one[0] == got[i]).all(), i


@pytest.mark.parametrize("offset", [0, 1, 3])
@pytest.mark.parametrize("rows,cols", [(131, 165), (257, 133)])
def test_any_alignment(zm, offset, rows, cols):
    x = matrices(10, 2, rows, cols)
    want, _ = run(zm, x, False)
    src = torch.zeros(x.size + 8, device=dev())
    src[offset:offset + x.size] = to_dev_f32(x.reshape(-1))
    out = torch.full((x.size + 8,), 7, dtype=torch.int16, device=dev())
    zm.zero_orthogonalize(src[offset:offset + x.size], out[offset:offset + x.size], rows, cols)
    got = host_u16(out)
    assert (got[offset:offset + x.size].reshape(x.shape) == want).all()
    assert (got[:offset] == 7).all() and (got[offset + x.size:] == 7).all()


@pytest.mark.parametrize("clip", [0.25, 1.0, float("nan"), float("inf"), float("-inf")])
@pytest.mark.parametrize("rows,cols", SIDES)
def test_clip(zm, clip, rows, cols):
    """A finite one scales the gradient; another skips the update and leaves everything as it was."""
    s = state(3, 2 * rows * cols)
    d = on_device(s)
    c = torch.full((1,), clip, device=dev())
    zm.zero_muon_step(*d, rows, cols, scale=3.0, clip_scale=c, **HYPER)
    if np.isfinite(clip):
        same(d, composed(zm, s, rows, cols, {}, clip, 3.0), clip)
    else:
        assert (host_f32(d[0]) == s[0]).all() and (host_f32(d[1]) == s[1]).all() and not host_u16(d[3]).any()


def test_a_matrix_that_is_not_finite_among_others_of_a_list(zm):
    """Its master and momentum take what its gradient holds; the other matrices' bits do not change."""
    shapes = [(150, 260), (260, 150), (300, 140), (40, 30)]
    sizes = [r * c for r, c in shapes]
    s = [state(20 + k, n) for k, n in enumerate(sizes)]
    ends = []
    for bad in (False, True):
        d = [on_device(x) for x in s]
        if bad:
            d[1][2][7] = 0x7F80
        zm.MuonTable(*[[x[k] for x in d] for k in range(4)], shapes).step(**HYPER)
        ends.append(d)
    for k in (0, 2, 3):
        assert all(torch.equal(a, b) for a, b in zip(ends[0][k], ends[1][k])), k
    assert torch.isnan(ends[1][1][0]).all()


def test_a_list_on_both_sides_of_128(zm):
    """The short ones take the tiled form with the others: each as the step on it alone, within the tiled form's precision."""
    shapes = [(64, 768)] * 5 + [(129, 768), (40, 30), (300, 100), (1, 50)]
    s = [state(60 + k, r * c) for k, (r, c) in enumerate(shapes)]
    d = [on_device(x) for x in s]
    zm.MuonTable(*[[x[k] for x in d] for k in range(4)], shapes).step(**HYPER)
    for (rows, cols), x, was in zip(shapes, d, s):
        note(f"{rows} x {cols}")
        buf, u = oracle.muon.momentum(was[1], was[2], HYPER["momentum"], True)
        o = oracle.muon.orthogonalize(u.reshape(rows, cols)).reshape(-1)
        rate = HYPER["lr"] * zm.muon_scale(rows, cols)
        want = was[0].astype(np.float64) * (1 - HYPER["lr"] * HYPER["weight_decay"]) - rate * o
        assert (host_f32(x[1]) == buf).all()
        off = np.linalg.norm(host_f32(x[0]) - want)
        assert off <= rate * FROBENIUS * np.linalg.norm(o) + 2 ** -23 * np.linalg.norm(want)
