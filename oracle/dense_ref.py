"""Dense products with bias, activation and residual, their gradients, and the
orthogonalised weight update in float64 (numpy): the formulas, nothing faster."""

from __future__ import annotations

import numpy as np
from scipy.special import erfc, expit

A, B, C = 3.4445, -4.7750, 2.0315


def act(z, name):
    if name == "relu":
        return np.where(z > 0, z, 0.0)
    if name == "gelu":
        return z * 0.5 * erfc(-z / np.sqrt(2.0))
    if name == "silu":
        return z * expit(z)
    return z


def slope(z, name):
    if name == "relu":
        return (z > 0).astype(np.float64)
    if name == "gelu":
        return 0.5 * erfc(-z / np.sqrt(2.0)) + z * np.exp(-z * z / 2) / np.sqrt(2 * np.pi)
    if name == "silu":
        return expit(z) * (1 + z * expit(-z))
    return np.ones_like(z)


def linear(x, w, bias=None, res=None, name="none"):
    """(y, z)"""
    z = x @ w.T
    if bias is not None:
        z = z + bias
    y = act(z, name)
    return (y if res is None else y + res), z


def linear_bwd(dy, x, w, z, name):
    """(dx, dw, dbias, dz)"""
    dz = dy if name == "none" else dy * slope(z, name)
    return dz @ w, dz.T @ x, dz.sum(axis=0), dz


def quintic(s):
    return A * s + B * s ** 3 + C * s ** 5


def orthogonalize(g, steps=5, eps=1e-7):
    """By the definition of the iteration on singular values: U p(...p(S)) V^T."""
    u, s, vt = np.linalg.svd(g, full_matrices=False)
    s = s / (np.sqrt((s * s).sum()) + eps)
    for _ in range(steps):
        s = quintic(s)
    return (u * s) @ vt


def iterate(g, steps=5, eps=1e-7, store=lambda v: v, mul=lambda a, b: a @ b):
    """The iteration as products, every stored matrix (X, A, B) through `store`
    and every product through `mul`: what a format's rounding does to it."""
    tall = g.shape[0] > g.shape[1]
    x = g.T if tall else g
    x = store(x / (np.sqrt((x * x).sum()) + eps))
    for k in range(steps):
        a = store(mul(x, x.T))
        b = store(A * np.eye(len(a)) + B * a + C * mul(a, a))
        x = mul(b, x)
        if k + 1 < steps:
            x = store(x)
    return x.T if tall else x


def store_f16(v):
    """fp16 after scaling by 2^13 (how the library keeps the iterates of bf16)."""
    return (v * 8192.0).astype(np.float16).astype(np.float64) / 8192.0


def store_2f16(v):
    """Two fp16 planes, hi + lo, after scaling by 2^13."""
    v = v * 8192.0
    hi = v.astype(np.float16).astype(np.float64)
    lo = (v - hi).astype(np.float16).astype(np.float64)
    return (hi + lo) / 8192.0


def mul_f32(a, b):
    """Products and sums in fp32."""
    return (a.astype(np.float32) @ b.astype(np.float32)).astype(np.float64)


def muon(w, g, buf, step, decay, mu, nesterov, steps=5, eps=1e-7, ortho=orthogonalize):
    """(w, buf)"""
    buf = mu * buf + g
    u = g + mu * buf if nesterov else buf
    return w * (1 - decay) - step * ortho(u, steps, eps), buf
