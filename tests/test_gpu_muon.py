"""The Muon operators on the GPU against the 64-bit oracle.

Tolerances. The result is rounded to bf16 once: at most 2^-8 of each value, in the 2-norm 2^-8 / sqrt(3) = 2.3e-3 where the
roundings are spread over a step. Before that each stored matrix is rounded to fp16, 2^-11 / sqrt(3) = 2.8e-4 of its norm. Of
a step those of X, A and C reach the next X by the factors p + 2 x p' (at most 2), b + 2 c x (at most 4.8 times A X) and 1:
together about 1.5e-3 of its norm, and three steps' (the earlier ones are damped) 2.6e-3. FROBENIUS holds the sum in
quadrature with half as much again; a single value can be 8 times the rms error off besides its own rounding.
Values of small matrices are not spread: those are held to the element bound only.
X after the first steps, whose values reach 1.23, is held as 2^13 of its value (the largest then lies in (2^13, 2^14]) in
fp16, whose step is 2^-24 at least: a value of it is off by up to 2^-38, which the steps that are left carry to the result with a^3 = 40.9, a^2 = 11.9 and a = 3.4: LEAST holds their sum. It
matters only where the norm is far below eps.
"""
import numpy as np
import pytest
import torch

import oracle
from tests.gpu_util import dev, host_f32, host_u16, needs_gpu, note, to_dev_f32, to_dev_u16

pytestmark = [pytest.mark.gpu, needs_gpu]

FROBENIUS = 5e-3
LEAST = 60 * 2.0 ** -38
STEPS = oracle.muon.COEFFICIENTS


@pytest.fixture(scope="module")
def zm():
    import zero_partitioned_mixed_partition_amd as m
    return m


def matrices(seed, count, rows, cols, size=1e-3, strong=8):
    """A few strong directions over noise."""
    rng = np.random.default_rng(seed)
    x = rng.normal(size=(count, rows, cols))
    k = min(strong, rows, cols)
    if k:
        x += 0.5 * (rng.normal(size=(count, rows, k)) * 2.0 ** (-np.arange(k) / 2)) @ rng.normal(size=(count, k, cols))
    return (x * size).astype(np.float32)


def check(got_bits, want, what):
    """got_bits [count, rows, cols] of bf16 against float64 of the same shape."""
    for i, (g, w) in enumerate(zip(oracle.bf16_to_f32(got_bits).astype(np.float64), want)):
        norm = np.linalg.norm(w)
        off = np.abs(g - w)
        rms = norm / np.sqrt(w.size)
        assert (off <= 2.0 ** -8 * np.abs(w) + 8 * 4e-3 * rms).all(), (what, i, (off - 2.0 ** -8 * np.abs(w)).max() / rms)
        if w.size >= 256:
            assert np.linalg.norm(off) <= FROBENIUS * norm, (what, i, np.linalg.norm(off) / norm)


def run(zm, x, bf16, **kw):
    """zero_orthogonalize of float32 [count, rows, cols] (rounded to bf16 first where bf16), and what went in."""
    count, rows, cols = x.shape
    if bf16:
        bits = oracle.f32_to_bf16(x)
        d, x = to_dev_u16(bits.reshape(-1)), oracle.bf16_to_f32(bits)
    else:
        d = to_dev_f32(x.reshape(-1))
    out = torch.full((x.size + 64,), 0x55, dtype=torch.int16, device=dev())
    zm.zero_orthogonalize(d, out[:x.size], rows, cols, **kw)
    got = host_u16(out)
    assert (got[x.size:] == 0x55).all(), "written past the end"
    return got[:x.size].reshape(x.shape), x


SHAPES = [(1, 1, 1), (1, 1, 7), (1, 7, 1), (3, 2, 3), (2, 5, 64), (1, 63, 65), (2, 64, 64), (1, 65, 63), (1, 127, 129), (1, 128, 128),
          (4, 129, 40), (1, 16, 1000), (1, 255, 257), (7, 33, 97), (1, 300, 1025), (1, 1025, 300), (2, 384, 640), (1, 520, 520),
          (12, 64, 768), (1, 1000, 512), (1, 3, 20000), (1, 20000, 2)]


@pytest.mark.parametrize("bf16", [True, False])
@pytest.mark.parametrize("shape", SHAPES)
def test_shapes(zm, shape, bf16):
    note(f"{shape} bf16={bf16}")
    got, x = run(zm, matrices(sum(shape), *shape), bf16)
    check(got, [oracle.muon.orthogonalize(m) for m in x], shape)


@pytest.mark.parametrize("count,rows,cols", [(1, 1536, 1600), (2, 700, 2100)])
def test_large(zm, count, rows, cols):
    got, x = run(zm, matrices(3, count, rows, cols), False)
    check(got, [oracle.muon.orthogonalize(m) for m in x], (rows, cols))


def on_gpu_in_64_bits(x, steps=STEPS, eps=1e-7):
    """The oracle's formula in float64 on the GPU, for sides whose products take a CPU too long."""
    if x.shape[0] > x.shape[1]:
        return on_gpu_in_64_bits(x.T.contiguous(), steps, eps).T
    x = x.double()
    x = x / (x.norm() + eps)
    for a, b, c in steps:
        gram = x @ x.T.contiguous()
        x = a * x + (b * gram + c * (gram @ gram)) @ x
    return x


@pytest.mark.parametrize("count,rows,cols", [(1, 2853, 3010), (1, 3010, 2853), (1, 4417, 4600), (9, 1030, 1100), (1, 2200, 2201), (3, 400, 5000),
                                             (1, 5950, 6001), (4, 2900, 2853)])
def test_tiles_that_end_inside_the_one_before(zm, count, rows, cols):
    """Sides that are no multiple of the tiles that such sizes take (the last two: tiles of which the last few are cut into
    quarters): each value is written once, by one workgroup."""
    note(f"{count} x {rows} x {cols}")
    x = to_dev_f32(matrices(7, count, rows, cols, strong=3).reshape(-1))
    out = [torch.full((x.numel() + 64,), 0x55, dtype=torch.int16, device=dev()) for _ in range(2)]
    for o in out:
        zm.zero_orthogonalize(x, o[:x.numel()], rows, cols)
    assert torch.equal(out[0], out[1]) and (out[0][x.numel():] == 0x55).all()
    got = out[0][:x.numel()].view(torch.bfloat16).view(count, rows, cols).double()
    for i in range(count):
        want = on_gpu_in_64_bits(x.view(count, rows, cols)[i])
        off = (got[i] - want).abs()
        rms = want.norm() / want.numel() ** 0.5
        assert (off <= 2.0 ** -8 * want.abs() + 8 * 4e-3 * rms).all(), i
        assert off.norm() <= FROBENIUS * want.norm(), (i, float(off.norm() / want.norm()))


@pytest.mark.parametrize("steps", [1, 2, 3, 4, 6, 9])
@pytest.mark.parametrize("shape", [(1, 96, 96), (2, 48, 400), (1, 400, 48)])
def test_step_counts(zm, shape, steps):
    got, x = run(zm, matrices(steps, *shape), False, coefficients=STEPS[:1] * steps)
    check(got, [oracle.muon.orthogonalize(m, STEPS[:1] * steps) for m in x], (shape, steps))


@pytest.mark.parametrize("rows,cols", [(33000, 70000), (70000, 33001)])
def test_past_2_to_the_31_elements(zm, rows, cols):
    """One value a row of the shorter side, each in a column of its own: they are the singular values, and the result is
    each one's polynomial in its place and zeros elsewhere."""
    note(f"{rows} x {cols}")
    m = min(rows, cols)
    gen = torch.Generator(device=dev()).manual_seed(1)
    values = (torch.rand(m, device=dev(), generator=gen) + 0.5).bfloat16()
    short = torch.arange(m, device=dev())
    at = short * cols + 2 * short + 1 if rows < cols else (2 * short + 1) * cols + short
    x = torch.zeros(rows * cols, dtype=torch.bfloat16, device=dev())
    x[at] = values
    out = torch.empty_like(x)
    zm.zero_orthogonalize(x, out, rows, cols)
    del x
    v = values.double()
    v = v / (v.norm() + 1e-7)
    for a, b, c in STEPS:
        v = a * v + b * v ** 3 + c * v ** 5
    got = out[at].double()
    # of a row's products all but one are of zeros: each step rounds X, A, C and what they make, as in the bound above
    assert ((got - v).abs() <= 2.0 ** -8 * v.abs() + 8 * 2.0 ** -11 * v.abs()).all(), float(((got - v) / v).abs().max())
    out[at] = 0
    assert not out.view(torch.int16).bitwise_and_(0x7fff).any()


@pytest.mark.parametrize("bf16", [True, False])
@pytest.mark.parametrize("steps", [1, 2, 3, 4, 7])
@pytest.mark.parametrize("shape", [(1, 150, 260), (1, 260, 150), (2, 200, 200)])
def test_step_counts_of_the_tiled_form(zm, shape, steps, bf16):
    """Sides past 128; with one step or two the first apply, which adds what rounding X left, is the last product."""
    got, x = run(zm, matrices(steps, *shape), bf16, coefficients=STEPS[:1] * steps)
    check(got, [oracle.muon.orthogonalize(m, STEPS[:1] * steps) for m in x], (shape, steps))


def test_other_coefficients(zm):
    """Steps of their own each, growing and shrinking, and one that is the identity."""
    steps = ((2.0, -1.5, 0.5), (1.5, -0.5, 0.0), (1.0, 0.0, 0.0), (1.875, -1.25, 0.375), (0.25, 0.0, 0.0))
    for n in (1, 3, 5):
        got, x = run(zm, matrices(n, 1, 90, 130), False, coefficients=steps[:n])
        check(got, [oracle.muon.orthogonalize(m, steps[:n]) for m in x], n)


@pytest.mark.parametrize("size", [1e-38, 1e-30, 1e-12, 1.0, 1e12, 1e30])
@pytest.mark.parametrize("eps", [0.0, 1e-7, 1.0])
def test_sizes_of_values(zm, size, eps):
    """Any magnitude fp32 holds; eps matters where the norm is near it."""
    x = matrices(5, 1, 40, 56, 1.0, strong=0)
    x = (x.astype(np.float64) * size).astype(np.float32)
    got, x = run(zm, x, False, eps=eps)
    want = [oracle.muon.orthogonalize(m, eps=eps) for m in x]
    if np.abs(want[0]).max() < 1e-6:        # norm far below eps
        w = np.abs(want[0])
        off = np.abs(oracle.bf16_to_f32(got[0]).astype(np.float64) - want[0])
        assert (off <= 2.0 ** -8 * w + 8 * 4e-3 * np.sqrt(np.mean(w * w)) + LEAST).all()
    else:
        check(got, want, (size, eps))


def test_zeros_infinities_and_nans_stay_in_their_matrix(zm):
    x = matrices(6, 7, 70, 90)
    clean, _ = run(zm, x, False)
    x[1] = 0.0
    x[2, 3, 4] = np.inf
    x[3, 69, 89] = -np.inf
    x[4, 0, 0] = np.nan
    x[5] = -0.0
    for eps in (1e-7, 0.0):
        got, _ = run(zm, x, False, eps=eps)
        f = oracle.bf16_to_f32(got)
        assert not f[1].any() and not f[5].any()
        assert np.isnan(f[2:5]).all()
    got, _ = run(zm, x, False)
    assert (got[[0, 6]] == clean[[0, 6]]).all()


def test_low_rank(zm):
    """Directions that the matrix does not have come out as noise of the stated size."""
    rng = np.random.default_rng(8)
    x = (rng.normal(size=(1, 200, 3)) @ rng.normal(size=(1, 3, 260))).astype(np.float32)
    got, x = run(zm, x, False)
    off = oracle.bf16_to_f32(got[0]).astype(np.float64) - oracle.muon.orthogonalize(x[0])
    assert np.linalg.norm(off, 2) < 0.02


def test_a_stack_is_its_matrices(zm):
    """Bit for bit, and the same bits twice."""
    x = matrices(9, 5, 100, 150)
    got, _ = run(zm, x, False)
    again, _ = run(zm, x, False)
    assert (got == again).all()
    for i in range(5):
        one, _ = run(zm, x[i:i + 1], False)
        assert (one[0] == got[i]).all(), i


@pytest.mark.parametrize("offset", [0, 1, 3])
def test_any_alignment(zm, offset):
    x = matrices(10, 2, 65, 131)
    want, _ = run(zm, x, False)
    src = torch.zeros(x.size + 8, device=dev())
    src[offset:offset + x.size] = to_dev_f32(x.reshape(-1))
    out = torch.full((x.size + 8,), 7, dtype=torch.int16, device=dev())
    zm.zero_orthogonalize(src[offset:offset + x.size], out[offset:offset + x.size], 65, 131)
    got = host_u16(out)
    assert (got[offset:offset + x.size].reshape(x.shape) == want).all()
    assert (got[:offset] == 7).all() and (got[offset + x.size:] == 7).all()


# ------------------------------------------------------------ the update

HYPER = dict(lr=4e-3, momentum=0.95, nesterov=True, weight_decay=0.1)


def state(seed, n):
    rng = np.random.default_rng(seed)
    return [rng.normal(size=n).astype(np.float32) * 0.02, rng.normal(size=n).astype(np.float32) * 5e-3,
            oracle.f32_to_bf16(rng.normal(size=n).astype(np.float32) * 1e-3)]


def on_device(s):
    return [to_dev_f32(s[0]), to_dev_f32(s[1]), to_dev_u16(s[2]), torch.zeros(len(s[0]), dtype=torch.int16, device=dev())]


def composed(zm, s, rows, cols, hyper, clip=1.0, scale=None, **kw):
    """Master, momentum and parameter bits from the formulas around zero_orthogonalize's bits."""
    h = dict(HYPER, **hyper)
    buf, u = oracle.muon.momentum(s[1], s[2], h["momentum"], h["nesterov"], clip)
    o, _ = run(zm, u.reshape(-1, rows, cols), False, **kw)
    scale = zm.muon_scale(rows, cols) if scale is None else scale
    p, bits = oracle.muon.apply(s[0], o.reshape(-1), h["lr"], scale, h["weight_decay"])
    return p, buf, bits


def same(d, want, what):
    p, buf, bits = want
    assert (host_f32(d[1]).view(np.uint32) == buf.view(np.uint32)).all(), (what, "momentum")
    assert (host_f32(d[0]).view(np.uint32) == p.view(np.uint32)).all(), (what, "master")
    assert (host_u16(d[3]) == bits).all(), (what, "param")


@pytest.mark.parametrize("count,rows,cols", [(1, 1, 1), (2, 30, 50), (1, 200, 77), (3, 128, 256), (1, 513, 300), (1, 64, 4000)])
@pytest.mark.parametrize("hyper", [{}, {"nesterov": False}, {"momentum": 0.0, "weight_decay": 0.0}, {"lr": 0.0}])
def test_step_is_momentum_orthogonalize_and_update(zm, count, rows, cols, hyper):
    s = state(rows, count * rows * cols)
    d = on_device(s)
    zm.zero_muon_step(*d, rows, cols, **dict(HYPER, **hyper))
    same(d, composed(zm, s, rows, cols, hyper), (rows, cols, hyper))


@pytest.mark.parametrize("count,rows,cols", [(1, 2853, 3010), (1, 4600, 4417), (9, 1030, 1100), (4, 2853, 2900)])
def test_a_step_with_large_tiles_updates_each_weight_once(zm, count, rows, cols):
    s = state(6, count * rows * cols)
    d = on_device(s)
    zm.zero_muon_step(*d, rows, cols, **HYPER)
    same(d, composed(zm, s, rows, cols, {}), (count, rows, cols))


def test_step_against_the_oracle(zm):
    """Three steps: what enters the master is lr * scale of the orthogonalised update, so it is off by that times its error."""
    rows, cols, n = 260, 190, 260 * 190
    s = state(1, n)
    d = on_device(s)
    master, buf = s[0].astype(np.float64), s[1]
    rate = HYPER["lr"] * zm.muon_scale(rows, cols)
    for t in range(3):
        grad = oracle.f32_to_bf16(np.random.default_rng(100 + t).normal(size=n).astype(np.float32) * 1e-3)
        d[2].copy_(to_dev_u16(grad))
        zm.zero_muon_step(*d, rows, cols, **HYPER)
        buf, u = oracle.muon.momentum(buf, grad, HYPER["momentum"], True)
        o = oracle.muon.orthogonalize(u.reshape(rows, cols))
        master = master * (1 - HYPER["lr"] * HYPER["weight_decay"]) - rate * o.reshape(-1)
    assert (host_f32(d[1]) == buf).all()
    off = np.linalg.norm(host_f32(d[0]) - master)
    assert off <= 3 * rate * FROBENIUS * np.linalg.norm(o) + 3 * 2 ** -23 * np.linalg.norm(master)
    assert (host_u16(d[3]) == oracle.f32_to_bf16(host_f32(d[0]))).all()


def test_clip_and_scale(zm):
    rows, cols = 90, 140
    s = state(2, rows * cols)
    for clip in (0.25, 1.0):
        d = on_device(s)
        zm.zero_muon_step(*d, rows, cols, scale=3.0, clip_scale=torch.full((1,), clip, device=dev()), **HYPER)
        same(d, composed(zm, s, rows, cols, {}, clip, 3.0), clip)


@pytest.mark.parametrize("clip", [float("nan"), float("inf"), float("-inf")])
def test_a_non_finite_clip_skips_the_update(zm, clip):
    rows, cols = 90, 140
    s = state(3, 2 * rows * cols)
    d = on_device(s)
    c = torch.full((1,), clip, device=dev())
    zm.zero_muon_step(*d, rows, cols, clip_scale=c, **HYPER)
    table = zm.MuonTable(*[[t] for t in d], [(rows, 2 * cols)])
    table.step(clip_scale=c, **HYPER)
    assert (host_f32(d[0]) == s[0]).all() and (host_f32(d[1]) == s[1]).all() and not host_u16(d[3]).any()


LIST = [(100, 60), (1, 33), (0, 5), (256, 256), (60, 100), (300, 40), (40, 300), (1, 1), (130, 131), (7, 513)]


@pytest.mark.parametrize("shift", [0, 1])
def test_a_table_is_its_matrices(zm, shift):
    """A ragged list in one arena, at odd places: each matrix as the step on it alone within the precision of the steps'
    grouping, the momenta bit for bit, and nothing between them written."""
    spans, at = [], shift
    for r, c in LIST:
        spans.append((at, r, c))
        at += r * c + 3
    s = state(4, at)
    d = on_device(s)
    cut = [[t[a:a + r * c] for a, r, c in spans] for t in d]
    table = zm.MuonTable(*cut, LIST)
    assert table.matrices == sum(1 for r, c in LIST if r * c)
    table.step(**HYPER)
    got = [host_f32(d[0]), host_f32(d[1]), host_u16(d[3])]
    gap = np.ones(at, bool)
    for a, r, c in spans:
        part = [x[a:a + r * c] for x in s]
        gap[a:a + r * c] = False
        if r * c == 0:
            continue
        p, buf, _ = composed(zm, part, r, c, {})
        assert (got[1][a:a + r * c] == buf).all(), (r, c)
        rate = HYPER["lr"] * zm.muon_scale(r, c)
        size = rate * np.sqrt(min(r, c)) * 1.2
        assert np.linalg.norm(got[0][a:a + r * c].astype(np.float64) - p) <= 2 * FROBENIUS * size, (r, c)
        assert (got[2][a:a + r * c] == oracle.f32_to_bf16(got[0][a:a + r * c])).all()
    assert (got[0][gap] == s[0][gap]).all() and (got[1][gap] == s[1][gap]).all() and not got[2][gap].any()


def test_a_table_of_one_is_the_step(zm):
    rows, cols = 170, 300
    s = state(5, rows * cols)
    a, b = on_device(s), on_device(s)
    zm.zero_muon_step(*a, rows, cols, **HYPER)
    zm.MuonTable(*[[t] for t in b], [(rows, cols)]).step(**HYPER)
    for x, y in zip(a, b):
        assert torch.equal(x, y)


def test_empty(zm):
    z = torch.zeros(0, device=dev())
    zb = torch.zeros(0, dtype=torch.int16, device=dev())
    zm.zero_muon_step(z, z, zb, zb, 0, 5, **HYPER)
    zm.zero_orthogonalize(z, zb, 5, 0)
    zm.MuonTable([], [], [], [], []).step(**HYPER)
    zm.MuonTable([z], [z], [zb], [zb], [(0, 4)]).step(**HYPER)
    torch.cuda.synchronize()


# ------------------------------------------------------------ streams and graphs

def test_two_streams_at_once(zm):
    """Each with a workspace of the call's own."""
    xs = [matrices(20 + k, 2, 300, 200) for k in range(2)]
    want = [run(zm, x, False)[0] for x in xs]
    src = [to_dev_f32(x.reshape(-1)) for x in xs]
    out = [torch.zeros(x.size, dtype=torch.int16, device=dev()) for x in xs]
    streams = [torch.cuda.Stream() for _ in xs]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    for _ in range(4):
        for k, s in enumerate(streams):
            zm.zero_orthogonalize(src[k], out[k], 300, 200, stream=s.cuda_stream)
    torch.cuda.synchronize()
    for k, x in enumerate(xs):
        assert (host_u16(out[k]).reshape(x.shape) == want[k]).all()


def test_graph_replays_are_successive_steps(zm):
    """A captured table step and a captured stack step, replayed with new gradients and eager work between, are the
    eager steps."""
    shapes = [(90, 200), (200, 90), (64, 64)]
    sizes = [r * c for r, c in shapes]
    s = [state(30 + k, n) for k, n in enumerate(sizes)]
    eager, graphed = [on_device(x) for x in s], [on_device(x) for x in s]
    table = zm.MuonTable(*[[d[k] for d in graphed] for k in range(4)], shapes)
    other = zm.MuonTable(*[[d[k] for d in eager] for k in range(4)], shapes)
    one = [on_device(state(40, 2 * 70 * 80)) for _ in range(2)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    ws = zm.muon_workspace(2, 70, 80, dev())
    prepared = table.prepare_step(stream=side.cuda_stream, **HYPER)
    with torch.cuda.graph(g, stream=side):
        prepared()
        zm.zero_muon_step(*one[0], 70, 80, workspace=ws, stream=side.cuda_stream, **HYPER)
    for t in range(4):
        for k, n in enumerate(sizes):
            grad = to_dev_u16(state(50 + 10 * t + k, n)[2])
            eager[k][2].copy_(grad)
            graphed[k][2].copy_(grad)
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        other.step(**HYPER)
        zm.zero_muon_step(*one[1], 70, 80, **HYPER)
        for a, b in zip(eager + one[1:], graphed + one[:1]):
            for x, y in zip(a, b):
                assert torch.equal(x, y), t
