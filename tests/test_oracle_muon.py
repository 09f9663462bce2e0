"""The Muon oracle against the singular values, closed forms and planted mistakes."""
import numpy as np
import pytest

from oracle import bf16, muon


@pytest.mark.parametrize("shape", [(1, 1), (1, 9), (9, 1), (5, 5), (7, 31), (40, 12)])
def test_the_products_are_the_polynomial_of_the_singular_values(shape):
    """Both forms in 64 bits: five steps of condition about 5 each on values of order 1, so well below 1e-9."""
    g = np.random.default_rng(1).normal(size=shape) * 1e-3
    np.testing.assert_allclose(muon.orthogonalize(g), muon.orthogonalize_by_svd(g), atol=1e-9)


def test_a_diagonal_matrix_step_by_step():
    s = np.array([0.5, 0.25, 0.1])
    x = s / (np.sqrt(np.sum(s * s)) + 1e-7)
    for a, b, c in muon.COEFFICIENTS:
        x = a * x + b * x ** 3 + c * x ** 5
    np.testing.assert_allclose(muon.orthogonalize(np.diag(s)), np.diag(x), atol=1e-12)
    assert (np.abs(x) > 0.65).all() and (np.abs(x) < 1.25).all()


def test_rotations_pass_through():
    rng = np.random.default_rng(2)
    g = rng.normal(size=(6, 11))
    u, v = np.linalg.qr(rng.normal(size=(6, 6)))[0], np.linalg.qr(rng.normal(size=(11, 11)))[0]
    np.testing.assert_allclose(muon.orthogonalize(u @ g @ v), u @ muon.orthogonalize(g) @ v, atol=1e-9)
    np.testing.assert_allclose(muon.orthogonalize(g.T), muon.orthogonalize(g).T, atol=1e-12)
    np.testing.assert_allclose(muon.orthogonalize(1e6 * g, eps=0.0), muon.orthogonalize(g, eps=0.0), atol=1e-12)


def test_zeros_and_non_finite_values():
    assert not muon.orthogonalize(np.zeros((3, 4))).any()
    assert not muon.orthogonalize(np.zeros((3, 4)), eps=0.0).any()
    for bad in (np.inf, np.nan):
        g = np.ones((3, 4))
        g[1, 2] = bad
        assert np.isnan(muon.orthogonalize(g)).all()


def test_the_update_by_hand():
    """Powers of two throughout: every result is exact."""
    grad = bf16.f32_to_bf16(np.array([2.0, -4.0], np.float32))
    buf, u = muon.momentum([1.0, 8.0], grad, 0.5, True, clip=0.5)
    assert buf.tolist() == [1.5, 2.0] and u.tolist() == [1.75, -1.0]
    assert muon.momentum([1.0, 8.0], grad, 0.5, False)[1].tolist() == [2.5, 0.0]
    p, bits = muon.apply([4.0, -2.0], bf16.f32_to_bf16(np.array([1.0, -0.5], np.float32)), 0.5, 2.0, 0.5)
    assert p.tolist() == [2.0, -1.0] and bf16.bf16_to_f32(bits).tolist() == [2.0, -1.0]


@pytest.mark.parametrize("mistake", ["sign", "order", "transpose", "norm"])
def test_planted_mistakes_are_seen(mistake):
    """A wrong formula in the oracle differs from the singular values' by far more than the two forms do."""
    g = np.random.default_rng(3).normal(size=(6, 9))
    x = g / (np.abs(g).max() if mistake == "norm" else np.linalg.norm(g))
    for a, b, c in muon.COEFFICIENTS[:2]:
        gram = x @ x.T
        if mistake == "sign":
            x = a * x - (b * gram + c * gram @ gram) @ x
        elif mistake == "order":
            x = a * x + (c * gram + b * gram @ gram) @ x
        elif mistake == "transpose":
            x = a * x + x @ (b * x.T @ x + c * gram[0, 0] * (x.T @ x))
        else:
            x = a * x + (b * gram + c * (gram @ gram)) @ x
    assert np.abs(x - muon.orthogonalize_by_svd(g, muon.COEFFICIENTS[:2])).max() > 1e-2
