"""The Muon entry points' argument checks, which all run before any HIP call (the addresses below are never
dereferenced), and the binding's."""
import ctypes

import pytest
import torch

FIVE = (ctypes.c_double * 15)(*((3.4445, -4.7750, 2.0315) * 5))
WS = 0x7000000000
MASTER, MOMENTUM, GRAD, PARAM = 0x1000000000, 0x2000000000, 0x3000000000, 0x4000000000


@pytest.fixture(scope="module")
def zm():
    import zero_partitioned_mixed_partition_amd as m
    return m


def _orth(zm, x=MASTER, kind=0, out=PARAM, count=2, rows=100, cols=200, steps=FIVE, n=5, eps=1e-7, ws=WS, size=1 << 40):
    return zm._binding._orth(x, kind, out, count, rows, cols, steps, n, eps, ws, size, None)


def _muon(zm, a=(MASTER, MOMENTUM, GRAD, PARAM), count=2, rows=100, cols=200, lr=1e-3, mu=0.95, wd=0.1, scale=2.0,
          steps=FIVE, n=5, eps=1e-7, ws=WS, size=1 << 40):
    return zm._binding._muon(*a, count, rows, cols, lr, mu, 1, wd, scale, steps, n, eps, None, ws, size, None)


@pytest.mark.parametrize("call", [_orth, _muon])
def test_refusals_of_both_forms(zm, call):
    b = zm._binding
    E, R, S, OK = b.ZERO_EINVAL, b.ZERO_ERANGE, b.ZERO_ENOSPACE, b.ZERO_OK
    for empty in (dict(count=0), dict(rows=0), dict(cols=0)):
        assert call(zm, **empty, ws=None, size=0) == OK
    for bad in (dict(count=-1), dict(rows=-1), dict(cols=-5), dict(n=0), dict(n=33), dict(steps=None), dict(eps=-1e-9),
                dict(eps=float("nan")), dict(eps=float("inf")), dict(ws=None), dict(ws=WS + 8)):
        assert call(zm, **bad) == E, bad
    for x in (float("nan"), float("inf")):
        assert call(zm, steps=(ctypes.c_double * 3)(1.0, x, 0.0), n=1) == E
    need = zm.zero_muon_workspace_bytes(2, 100, 200)
    assert call(zm, size=need - 1) == S and str(need) in zm.zero_last_error()
    assert call(zm, rows=65537, cols=65537) == R and call(zm, rows=1, cols=(1 << 22) + 1) == R
    assert call(zm, count=1 << 40) == R
    assert call(zm, steps=(ctypes.c_double * 3)(2.0 ** 30, 0.0, 0.0), n=1) == E and "2^20" in zm.zero_last_error()


def test_orthogonalize_refusals(zm):
    E = zm._binding.ZERO_EINVAL
    assert _orth(zm, kind=2) == E and _orth(zm, kind=-1) == E
    assert _orth(zm, x=None) == E and _orth(zm, out=None) == E
    for kind, size in ((0, 2), (1, 4)):                  # 2 x 100 x 200 elements
        assert _orth(zm, kind=kind, out=MASTER + 40000 * size - 2) == E and "out overlaps x" in zm.zero_last_error()
    assert _orth(zm, x=WS + 256) == E and "workspace overlaps x" in zm.zero_last_error()
    assert _orth(zm, out=WS + 256) == E and "out overlaps workspace" in zm.zero_last_error()


def test_step_refusals(zm):
    E = zm._binding.ZERO_EINVAL
    nan, inf = float("nan"), float("inf")
    for bad in (dict(lr=-1e-3), dict(lr=nan), dict(lr=inf), dict(mu=1.0), dict(mu=-0.1), dict(mu=nan), dict(wd=inf),
                dict(scale=nan), dict(scale=inf)):
        assert _muon(zm, **bad) == E, bad
    a = [MASTER, MOMENTUM, GRAD, PARAM]
    names, sizes = ("master", "momentum", "grad", "param_out"), (4, 4, 2, 2)
    for k in range(4):
        assert _muon(zm, a=a[:k] + [None] + a[k + 1:]) == E and "NULL array" in zm.zero_last_error()
        for j in range(4):
            if j == k:
                continue
            clash = list(a)
            clash[j] = a[k] + 40000 * sizes[k] - 2
            assert _muon(zm, a=clash) == E
            text = zm.zero_last_error()
            assert names[j] in text and names[k] in text and "overlaps" in text, text
        clash = list(a)
        clash[k] = WS + 4096
        assert _muon(zm, a=clash) == E and "workspace" in zm.zero_last_error()


def _create(zm, mats, n=None, drop=None, out=True, scales=None):
    """mats: (master, momentum, grad, param, rows, cols) each."""
    T = max(len(mats), 1)
    tabs = [(ctypes.c_void_p * T)(*[m[k] for m in mats]) for k in range(4)]
    sides = [(ctypes.c_int64 * T)(*[m[4 + k] for m in mats]) for k in range(2)]
    args = tabs + sides + [(ctypes.c_double * T)(*(scales or [1.0] * len(mats)))]
    if drop is not None:
        args[drop] = None
    h = ctypes.c_void_p()
    st = zm._binding._muont_create(*args, len(mats) if n is None else n, ctypes.byref(h) if out else None)
    return st, h


def test_table_refusals(zm):
    b = zm._binding
    E, R, OK = b.ZERO_EINVAL, b.ZERO_ERANGE, b.ZERO_OK
    one = (MASTER, MOMENTUM, GRAD, PARAM, 100, 200)
    far = tuple(x + 0x100000000 for x in one[:4]) + (30, 40)
    assert _create(zm, [one], out=False)[0] == E and _create(zm, [one], n=-1)[0] == E
    for k in range(7):
        assert _create(zm, [one], drop=k)[0] == E
    for k in range(4):
        assert _create(zm, [one, far[:k] + (None,) + far[k + 1:]])[0] == E
        assert "matrix 1 has a NULL array" in zm.zero_last_error()
    assert _create(zm, [one, far[:4] + (-1, 4)])[0] == E and "matrix 1 has a negative side" in zm.zero_last_error()
    assert _create(zm, [far[:4] + (1 << 17, 1 << 17)])[0] == R and _create(zm, [far[:4] + ((1 << 22) + 1, 1)])[0] == R
    assert _create(zm, [one], scales=[float("nan")])[0] == E
    for k in range(4):                                   # matrix 1's array k on matrix 0's master
        clash = far[:k] + (MASTER + 4,) + far[k + 1:]
        assert _create(zm, [one, clash])[0] == E and "master 0" in zm.zero_last_error(), zm.zero_last_error()
    shared = far[:2] + (GRAD,) + far[3:]                 # a gradient read twice is no clash: fails later, on the device
    assert "overlaps" not in (zm.zero_last_error() if _create(zm, [one, shared])[0] == E else "")


def test_empty_tables(zm):
    b = zm._binding
    for mats in ([], [(None, None, None, None, 0, 7)]):
        st, h = _create(zm, mats)
        assert st == b.ZERO_OK and b._muont_count(h) == 0 and b._muont_ws(h) == 0
        assert b._muont_step(h, 1e-3, 0.9, 1, 0.0, FIVE, 5, 1e-7, None, None, 0, None) == b.ZERO_OK
        for bad in ((-1.0, 0.9, 1, 0.0), (1e-3, 1.0, 1, 0.0), (1e-3, 0.9, 1, float("nan"))):
            assert b._muont_step(h, *bad, FIVE, 5, 1e-7, None, None, 0, None) == b.ZERO_EINVAL
        b._muont_free(h)
    assert b._muont_step(None, 1e-3, 0.9, 1, 0.0, FIVE, 5, 1e-7, None, None, 0, None) == b.ZERO_EINVAL
    assert b._muont_count(None) == -1 and b._muont_ws(None) == 0
    b._muont_free(None)


def test_workspace_bytes(zm):
    """0 where there is nothing to do or the sizes are refused; grows with each size."""
    w = zm.zero_muon_workspace_bytes
    for none in ((0, 5, 5), (5, 0, 5), (5, 5, 0), (-1, 5, 5), (1, 65537, 65537), (1, 1, (1 << 22) + 1)):
        assert w(*none) == 0
    assert 0 < w(1, 1, 1) <= w(1, 100, 200) < w(2, 100, 200) and w(1, 100, 200) == w(1, 200, 100)
    assert w(1, 1000, 2000) >= 8 * 1000 * 2000 + 6 * 1000 * 1000


def test_binding_refusals(zm):
    x = torch.zeros(12, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="no stack of 5 x 2"):
        zm.zero_orthogonalize(x, x, 5, 2)
    with pytest.raises(ValueError, match="no stack of 0 x 2"):
        zm.zero_orthogonalize(x, x, 0, 2)
    with pytest.raises(ValueError, match="negative"):
        zm.zero_orthogonalize(x, x, -3, -4)
    with pytest.raises(ValueError, match="not torch.float16"):
        zm.zero_orthogonalize(x.half(), x, 3, 4)
    with pytest.raises(ValueError, match="not torch.float16"):
        zm.zero_orthogonalize(x, x.half(), 3, 4)
    with pytest.raises(ValueError, match="not torch.float64"):
        zm.zero_orthogonalize(x.double(), x, 3, 4)
    with pytest.raises(ValueError, match="out holds 11"):
        zm.zero_orthogonalize(x, x[:11], 3, 4)
    with pytest.raises(ValueError, match="device tensor"):
        zm.zero_orthogonalize(x, x.clone(), 3, 4)
    with pytest.raises(ValueError, match="device tensor"):
        zm.zero_muon_step(x.float(), x.float(), x, x.clone(), 3, 4, 1e-3)
    with pytest.raises(ValueError, match="same length"):
        zm.MuonTable([x], [x], [x], [], [(3, 4)])
    with pytest.raises(ValueError, match="same length"):
        zm.MuonTable([x], [x], [x], [x], [(3, 4)], scales=[])
    zm.zero_orthogonalize(x[:0], x[:0], 0, 4)            # nothing to do
    assert zm.muon_scale(100, 25) == pytest.approx(2.0)
