"""Muon in 64 bits: the orthogonalisation by Newton-Schulz steps from its formula, and the update of a weight matrix.

Written from the mathematics alone, over numpy float64: per step, X <- a X + (b A + c A^2) X with A = X X^T. The
orthogonalised update is held in bf16 where the weight update uses it, and the update itself is one fp32 operation at
a time.
"""
from __future__ import annotations

import numpy as np

from . import bf16

COEFFICIENTS = ((3.4445, -4.7750, 2.0315),) * 5


def orthogonalize(g, coefficients=COEFFICIENTS, eps: float = 1e-7) -> np.ndarray:
    """float64 [rows, cols] of a matrix, unrounded."""
    x = np.asarray(g, np.float64)
    if x.shape[0] > x.shape[1]:
        return orthogonalize(x.T, coefficients, eps).T
    norm = np.sqrt(np.sum(x * x))
    if norm == 0.0:
        return np.zeros_like(x)
    with np.errstate(invalid="ignore", over="ignore"):
        x = x / (norm + eps)
        for a, b, c in coefficients:
            gram = x @ x.T
            x = a * x + (b * gram + c * (gram @ gram)) @ x
    return x


def orthogonalize_by_svd(g, coefficients=COEFFICIENTS, eps: float = 1e-7) -> np.ndarray:
    """The same through the singular values: each step is an odd polynomial of them."""
    x = np.asarray(g, np.float64)
    u, s, vt = np.linalg.svd(x, full_matrices=False)
    s = s / (np.sqrt(np.sum(s * s)) + eps)
    for a, b, c in coefficients:
        s = a * s + b * s ** 3 + c * s ** 5
    return (u * s) @ vt


def momentum(buf, grad_bits, mu: float, nesterov: bool, clip: float = 1.0):
    """The new momentum and the matrix to orthogonalise, in fp32, one operation at a time. grad_bits: uint16."""
    f = np.float32
    g = bf16.bf16_to_f32(np.asarray(grad_bits, np.uint16)) * f(clip)
    buf = f(mu) * np.asarray(buf, f) + g
    return buf, (g + f(mu) * buf if nesterov else buf)


def apply(master, o_bits, lr: float, scale: float, weight_decay: float):
    """The new fp32 master and bf16 parameter bits from the orthogonalised update's bf16 bits."""
    f = np.float32
    p = np.asarray(master, f) * f(1.0 - lr * weight_decay)
    p = p - f(lr * scale) * bf16.bf16_to_f32(np.asarray(o_bits, np.uint16))
    return p, bf16.f32_to_bf16(p)
