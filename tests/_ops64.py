"""The operators around the GEMM in 64 bits, from their definitions (numpy; activations
through scipy's normal distribution function), and the bounds on the fp32 kernels' distance
from them. Test infrastructure.

Each bound is a count of fp32 roundings (u = 2^-24 relative each) of the formula as the
kernels evaluate it, rounded up to a power of two; the output's own rounding comes on top."""
from __future__ import annotations

import numpy as np
from scipy.special import expit, ndtr

U = 2.0 ** -24
ACTS = ("none", "relu", "silu", "gelu", "gelu_tanh")
C_TANH = np.sqrt(2 / np.pi)


def act(z, name):
    z = np.asarray(z, dtype=np.float64)
    if name == "relu":
        return np.maximum(z, 0.0)
    if name == "silu":
        return z * expit(z)
    if name == "gelu":
        return z * ndtr(z)
    if name == "gelu_tanh":
        return z * expit(2 * C_TANH * (z + 0.044715 * z ** 3))
    return z


def act_slope(z, name):
    z = np.asarray(z, dtype=np.float64)
    if name == "relu":
        return (z > 0).astype(np.float64)
    if name == "silu":
        s = expit(z)
        return s * (1 + z * (1 - s))
    if name == "gelu":
        return ndtr(z) + z * np.exp(-z * z / 2) / np.sqrt(2 * np.pi)
    if name == "gelu_tanh":
        s = expit(2 * C_TANH * (z + 0.044715 * z ** 3))
        return s + z * s * (1 - s) * 2 * C_TANH * (1 + 3 * 0.044715 * z * z)
    return np.ones_like(z)


def act_bound(z, dz, name):
    """|act in fp32 of (z +- dz) - act(z)|. |act'| <= 1.13 carries dz over. The rest: a few
    roundings, the polynomial's 2^-25, and the exponent of e^-z, e^(-z^2/2) or e^(2u), whose
    argument of size up to 1 + |z| + z^2 (gelu_tanh: 2 (|z| + |z|^3 / 22)) is off by a few u
    and so the power by as many times u; below 2^-126 the power flushes to zero."""
    if name in ("none", "relu"):
        return dz
    a = np.abs(z)
    arg = 1 + a + a * a if name != "gelu_tanh" else 2 + 2 * a + a ** 3 / 8
    return 1.13 * dz + np.abs(act(z, name)) * (2.0 ** -20 + 4 * U * arg) + 2.0 ** -120


def slope_bound(z, name):
    """|act' in fp32 - act'(z)|: terms of size up to 2 with the relative errors of act_bound,
    where the terms that the exponent's error multiplies decay with the power itself."""
    return 0.0 if name in ("none", "relu") else 2.0 ** -19


def rmsnorm(x, r, w, eps):
    """(y, s, rstd) in fp64."""
    s = np.asarray(x, dtype=np.float64) + (0 if r is None else np.asarray(r, dtype=np.float64))
    rstd = 1 / np.sqrt(np.mean(s * s, axis=1) + eps)
    return s * rstd[:, None] * np.asarray(w, dtype=np.float64), s, rstd


# rstd: 32 sequential squares per thread, 6 + 16 tree and wave additions, all of one sign:
# 54 u on the sum, halved by the root, and 5 roundings after it
RSTD_REL = 2.0 ** -18
# y: rstd's, the rounding of x + r, two products
Y_REL = 2.0 ** -17


def rmsnorm_backward(dy, h, w, rstd, dh=None):
    """(dx, dweight, bound on dx, bound on dweight) in fp64, from the stored h and rstd.
    Bounds: the row's mean is a sum of K products in 64 additions deep (2^-17 of the sum of
    magnitudes); the column sums are at most 200 rows and partials deep (2^-16)."""
    dy, h, w = (np.asarray(t, dtype=np.float64) for t in (dy, h, w))
    q = np.asarray(rstd, dtype=np.float64)[:, None]
    xh, g = h * q, dy * w
    mean = np.mean(g * xh, axis=1, keepdims=True)
    dx = q * (g - xh * mean)
    mag = q * (np.abs(g) + np.abs(xh) * np.mean(np.abs(g * xh), axis=1, keepdims=True))
    bound = 2.0 ** -17 * mag
    if dh is not None:
        dx = dx + np.asarray(dh, dtype=np.float64)
        bound = bound + 2 * U * np.abs(dh)
    return dx, (dy * xh).sum(0), bound, 2.0 ** -16 * np.abs(dy * xh).sum(0)


def bf16_slack(x):
    """Half a bf16 ulp at |x| (8 significant bits)."""
    return 2.0 ** -8 * np.abs(x) + 2.0 ** -134
