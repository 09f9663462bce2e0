"""The products and scalings that the Muon planner makes for coefficients, on the CPU (tests/host_muon_program.cpp prints
them): which coefficients it takes, and that no value it holds leaves fp16's range."""
import math
import os
import shutil
import subprocess

import numpy as np
import pytest

import oracle

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "zero_partitioned_mixed_partition_amd", "csrc")
ROCM = os.environ.get("ROCM_PATH", "/opt/rocm")

pytestmark = pytest.mark.skipif(shutil.which("g++") is None or not os.path.exists(f"{ROCM}/include/hip"),
                                reason="needs g++ and the HIP headers")

# The published Polar Express steps: each contracts to the very end of the interval that the one before leaves, and
# grows steeply past it.
POLAR = ((8.28721201814563, -23.595886519098837, 17.300387312530933), (4.107059111542203, -2.9478499167379106, 0.5448431082926601),
         (3.9486908534822946, -2.908902115962949, 0.5518191394370137), (3.3184196573706015, -2.488488024314874, 0.51004894012372),
         (2.300652019954817, -1.6689039845747493, 0.4188073119525673))
USUAL = oracle.muon.COEFFICIENTS[0]
MARGIN = 65504 / 2 ** 14         # what fp16 holds past the planned bound, which lies in (2^13, 2^14]


def divided(steps, s):
    return [(a / s, b / s ** 3, c / s ** 5) for a, b, c in steps]


@pytest.fixture(scope="module")
def exe(tmp_path_factory):
    out = str(tmp_path_factory.mktemp("muon") / "program")
    b = subprocess.run(["g++", "-O1", "-g", "-std=c++17", "-fsanitize=address,undefined", "-fno-sanitize-recover=all",
                        f"-I{ROCM}/include", "-D__HIP_PLATFORM_AMD__", f"-I{CSRC}",
                        f"-I{os.path.join(ROOT, 'include')}", os.path.join(ROOT, "tests", "host_muon_program.cpp"),
                        os.path.join(CSRC, "muon_plan.cpp"), os.path.join(CSRC, "status.cpp"), "-o", out,
                        f"-L{ROCM}/lib", "-lamdhip64", f"-Wl,-rpath,{ROCM}/lib"], capture_output=True, text=True, timeout=300)
    assert b.returncode == 0, b.stderr[-2000:]
    return out


def run(exe, *args, steps):
    r = subprocess.run([exe, *args, *[repr(float(x)) for s in steps for x in s]], capture_output=True, text=True, timeout=60,
                       env=dict(os.environ, ASAN_OPTIONS="detect_leaks=0"))
    assert r.returncode == 0, r.stderr
    return r.stdout.splitlines()


def tiled(exe, steps, pairs, low):
    """Status, message, and the products as (kind, lhs, rhs, add, out, kappa power, low in, low out, full, alpha, beta, diag)."""
    head, *rows = run(exe, "tiled", str(int(pairs)), str(int(low)), steps=steps)
    status, _, message = head.partition(" ")
    return int(status), message, [[int(x) for x in r.split()[:9]] + [float(x) for x in r.split()[9:]] for r in rows]


GRAM, SQUARE, APPLY, FINAL = range(4)


def held(x):
    """fp16 of x, which must stay in its range."""
    with np.errstate(over="ignore"):
        h = x.astype(np.float16).astype(np.float64)
    assert np.isfinite(h).all(), "a held value left fp16's range"
    return h


def emulate(products, g, eps=1e-7):
    """The tiled form's products on a matrix with rows <= cols: every held value in fp16, sums in 64 bits."""
    norm = np.sqrt(np.sum(g * g))
    e = math.frexp(norm)[1] - 1
    kappa = 2.0 ** (e + 1) / (norm + eps)
    u = g * 2.0 ** (13 - e)
    x = held(u)
    rest = held(u - x)
    s = {}
    for kind, lhs, rhs, add, out, power, low_in, low_out, full, alpha, beta, diag in products:
        alpha *= kappa ** power
        if kind == GRAM:
            s[out] = held(alpha * (x @ x.T))
        elif kind == SQUARE:
            v = alpha * (s[lhs] @ s[rhs].T) + diag * np.eye(len(x))
            if beta:
                v += beta * s[add]
            if not full:                                     # computed on the tiles at and below the diagonal, mirrored
                tile = np.arange(len(v)) // 64
                v = np.where(tile[:, None] >= tile, v, v.T)
            s[out] = held(v)
        else:
            v = s[lhs] @ x
            if low_in:
                v += np.diag(s[lhs])[:, None] * rest
            v *= alpha
            if kind == FINAL:
                assert not low_out
                return v
            x = held(v)
            rest = held(v - x) if low_out else None


def matrix(kind, m=40, n=70):
    rng = np.random.default_rng(len(kind))
    if kind == "gradient":
        return rng.normal(size=(m, n)) + 0.5 * (rng.normal(size=(m, 8)) * 2.0 ** (-np.arange(8) / 2)) @ rng.normal(size=(8, n))
    if kind == "row":
        return rng.normal(size=(1, n))
    if kind == "rank one":
        return rng.normal(size=(m, 1)) @ rng.normal(size=(1, n))
    if kind == "diagonal":                                   # every singular value an element of its own
        return np.eye(m, n) * rng.uniform(0.05, 1.0, size=(m, 1))
    u, v = np.linalg.qr(rng.normal(size=(m, m)))[0], np.linalg.qr(rng.normal(size=(n, m)))[0]
    return (u * np.linspace(0.02, 1.0, m)) @ v.T


SAFETY = 1 + 3 * 2.0 ** -11
EDGE = {"published": POLAR, "rounded to three digits": [tuple(round(x, 3) for x in s) for s in POLAR], "four": POLAR[:4],
        "over 1.001": divided(POLAR, 1.001)}
AS_GIVEN = {"over 1.003": divided(POLAR, 1.003), "over 1.01, but the last": divided(POLAR[:4], 1.01) + [POLAR[4]], "one": POLAR[:1],
            "usual": [USUAL] * 5, "usual, nine": [USUAL] * 9}


@pytest.mark.parametrize("pairs", [False, True])
@pytest.mark.parametrize("name", [*EDGE, *AS_GIVEN])
def test_steps_that_end_at_the_edge_of_their_interval(exe, name, pairs):
    """They are taken, nothing that is held leaves its range, and the result is that of the steps with X a little smaller
    (SAFETY) in all but the last, or, where they contract past the edge, of the steps as they are.

    Tolerance: a step's roundings are 1.5e-3 of X's norm (test_gpu_muon.py); the steps that follow magnify what they leave
    of a value near 1 by their slope there, 5 at most for these sets (the published set's oscillates so, the usual one's is
    below 2), so 7.5e-3 a step and, the earlier ones damped, 2e-2. Matrices of few directions are not held to it: their
    largest singular value only, which is what a wrong interval lets grow."""
    given = EDGE.get(name) or AS_GIVEN[name]
    taken = divided(given[:-1], SAFETY) + [given[-1]] if name in EDGE else given
    status, message, products = tiled(exe, given, pairs, True)
    assert status == 0, message
    for kind in ("gradient", "spread", "diagonal", "row", "rank one"):
        g = matrix(kind)
        got, want = emulate(products, g), oracle.muon.orthogonalize(g, taken)
        assert np.linalg.norm(got, 2) <= 1.05 * np.linalg.norm(want, 2) + 0.02, kind
        if kind != "rank one" and name != "usual, nine":
            assert np.linalg.norm(got - want) <= 2e-2 * np.linalg.norm(want), (kind, np.linalg.norm(got - want))


@pytest.mark.parametrize("steps", [[(1.0, 1.0, 1.0)] * 6, [(2.0 ** 30, 0.0, 0.0)], [(8.0, 0.0, 0.0)] * 8, [(3.0, 2.0, 0.0)] * 5])
def test_steps_that_grow_are_refused(exe, steps):
    status, message, _ = tiled(exe, steps, False, True)
    assert status != 0 and "grow past 2^20" in message


@pytest.mark.parametrize("pairs", [False, True])
@pytest.mark.parametrize("steps", [[(1e308, 1e308, 1e308)], [(1e308, -1e308, 1e308)] * 2, [(0.0, 0.0, 0.0), (1e200, 0.0, 0.0)],
                                   [(1e-30, 0.0, 0.0), USUAL, (-1e60, 1e80, 0.0), USUAL]])
def test_factors_past_any_exponent_are_refused(exe, steps, pairs):
    """With the address and undefined-behaviour checks of the compiler."""
    status, message, _ = tiled(exe, steps, pairs, True)
    assert status != 0 and ("grow past 2^20" in message or "more than 2^60" in message)
    assert short(exe, steps) is None


SPECTRA = {"rank 1": lambda k, m: (k < 1) * 1.0, "rank 3": lambda k, m: (k < 3) * 1.0, "flat": lambda k, m: np.ones(m),
           "32 over 1e-3": lambda k, m: np.where(k < 32, 1.0, 1e-3), "8 over 1e-4": lambda k, m: np.where(k < 8, 1.0, 1e-4),
           "half over 1e-3": lambda k, m: np.where(k < m // 2, 1.0, 1e-3), "1/k^2": lambda k, m: (1.0 + k) ** -2.0,
           "1e-3 by ratios": lambda k, m: 10.0 ** (-3 * k / m), "1e-6 by ratios": lambda k, m: 10.0 ** (-6 * k / m)}


@pytest.mark.parametrize("fp32", [True, False])
@pytest.mark.parametrize("pairs", [False, True])
@pytest.mark.parametrize("kind", list(SPECTRA))
def test_what_rounding_x_leaves_is_carried_along(exe, kind, pairs, fp32):
    """Hard singular values in random directions: FIVE of tests/test_gpu_muon_spectra.py (derived there), without bf16's
    rounding."""
    m, n = 150, 260
    rng = np.random.default_rng(1)
    u, v = np.linalg.qr(rng.normal(size=(m, m)))[0], np.linalg.qr(rng.normal(size=(n, m)))[0]
    g = (u * SPECTRA[kind](np.arange(m), m)) @ v.T
    g = (g.astype(np.float32) if fp32 else oracle.bf16_to_f32(oracle.f32_to_bf16(g.astype(np.float32)))).astype(np.float64)
    _, _, products = tiled(exe, [USUAL] * 5, pairs, fp32)
    want = oracle.muon.orthogonalize(g)
    assert np.linalg.norm(emulate(products, g) - want) <= 6.6e-3 * np.linalg.norm(want)


def short(exe, steps):
    head, *rows = run(exe, "short", steps=steps)
    return [[float(x) for x in r.split()] for r in rows] if head == "1" else None


def test_short_sides_take_the_usual_steps_and_leave_steep_ones(exe):
    """Steps whose roundings grow too far in directions that the matrix does not have go to the tiled form."""
    for n in (1, 5):
        assert short(exe, [USUAL] * n) is not None
    assert short(exe, [(2.0, -1.5, 0.5), (1.5, -0.5, 0.0), (1.0, 0.0, 0.0)]) is not None
    assert short(exe, [USUAL] * 9) is None and short(exe, POLAR) is None


def test_what_short_sides_hold_stays_in_range(exe):
    """Random steps that are taken: A, C, T and Q, at eigenvalues far denser than the planner's, within fp16's range."""
    rng = np.random.default_rng(0)
    x0 = np.concatenate([np.linspace(0.0, 1.0, 200001), np.logspace(-12, 0, 200001)])
    taken = 0
    for _ in range(60):
        steps = [USUAL] * rng.integers(0, 4) + [(rng.uniform(0.5, 4.0), rng.uniform(-6.0, 0.5), rng.uniform(-0.5, 4.0))
                                                for _ in range(rng.integers(1, 4))]
        rows = short(exe, steps)
        if rows is None:
            continue
        taken += 1
        x, q = x0.copy(), np.ones_like(x0)
        hold_a, hold_q = rows[0][0], 1.0
        for k, ((a, b, c), (ha, hb, hc, t, nxt, hq)) in enumerate(zip(steps, rows[1:])):
            hold_c = ha / a
            p = a + x * (b + x * c)
            assert np.abs(x).max() * hold_a <= 65504 and np.abs(p).max() * hold_c <= 65504, steps
            assert np.abs(x * p).max() * hold_a * hold_c * t <= 65504, steps
            q = q * p
            hold_q = hold_c if k == 0 else hold_q * hold_c * hq
            assert np.abs(q).max() * hold_q <= 65504, steps
            x = x * p * p
            hold_a = hold_a * hold_c * hold_c * t * nxt
    assert taken >= 15
