"""Layer norm, gated product and dropout in 64 bits, from their definitions, and the bounds on
the fp32 kernels' distance from them. Test infrastructure; the conventions of _ops64.

Sums over a row of K <= 32768 values: at most 64 sequential additions in a thread, 6 in the
wave, 8 over the waves and a few roundings, below 128 u = 2^-17 of the sum of magnitudes.
Column sums are at most 200 rows and partials deep: 2^-16."""
from __future__ import annotations

import numpy as np

from tests import _ops64 as ops

U = ops.U
ROW, COL = 2.0 ** -17, 2.0 ** -16


def philox(counter, key, rounds=7):
    """Philox 4x32: counter (four arrays or numbers) and key (two) to four arrays, uint64."""
    u = np.uint64
    c = [np.atleast_1d(np.asarray(v, dtype=u)) for v in counter]
    k = [int(v) for v in key]
    low, half = u(0xFFFFFFFF), u(32)
    for _ in range(rounds):
        a, b = u(0xD2511F53) * c[0], u(0xCD9E8D57) * c[2]
        c = [(b >> half) ^ c[1] ^ u(k[0]), b & low, (a >> half) ^ c[3] ^ u(k[1]), a & low]
        k = [(k[0] + 0x9E3779B9) & 0xFFFFFFFF, (k[1] + 0xBB67AE85) & 0xFFFFFFFF]
    return c


def threshold(p):
    return int(65536 * p + 0.5)


def kept(first, n, p, seed, offset, subsequence=0):
    """Truth values of elements first .. first + n - 1 (first a multiple of 8)."""
    o = (offset + subsequence) & 0xFFFFFFFFFFFFFFFF
    seed &= 0xFFFFFFFFFFFFFFFF
    g = np.arange(first // 8, (first + n + 7) // 8, dtype=np.uint64)
    w = philox((g & np.uint64(0xFFFFFFFF), g >> np.uint64(32), np.full_like(g, o & 0xFFFFFFFF), np.full_like(g, o >> 32)),
               (seed & 0xFFFFFFFF, seed >> 32))
    bits = np.stack([h for v in w for h in (v & np.uint64(0xFFFF), v >> np.uint64(16))], 1)
    return bits.reshape(-1)[:n] >= threshold(p)


def dropout(x, p, seed, offset, subsequence=0):
    x = np.asarray(x, dtype=np.float64)
    t = threshold(p)
    if t == 0:
        return x
    return np.where(kept(0, x.size, p, seed, offset, subsequence).reshape(x.shape), x * (65536 / (65536 - t)), 0.0)


def sum_before_norm(x, r, p=0.0, seed=0, offset=0, subsequence=0):
    """(s, bound): the factor's and the product's rounding where there is dropout, the sum's."""
    d = dropout(x, p, seed, offset, subsequence)
    s = d if r is None else d + np.asarray(r, dtype=np.float64)
    return s, (2 * U * np.abs(d) if threshold(p) else 0) + (U * np.abs(s) if r is not None else 0) + 0 * s


def layernorm(s, es, w, b, eps):
    """y, mean, rstd and bounds on them, s known to es. With m the rounding of a mean (of a wave's
    values or of the row's): the variance is off by its own roundings, by m^2 and 2 m deviation
    (squares about a mean that is m off), and by what es moves; rstd by half of that."""
    s, w = np.asarray(s, dtype=np.float64), np.asarray(w, dtype=np.float64)
    mean = s.mean(1, keepdims=True)
    d = s - mean
    var = (d * d).mean(1, keepdims=True)
    rstd = (var + eps) ** -0.5
    size = np.abs(s).mean(1, keepdims=True)
    dmean = ROW * size + np.mean(es, axis=1, keepdims=True)
    dev, e = np.sqrt(var), np.sqrt(np.mean(np.broadcast_to(es, s.shape) ** 2, axis=1, keepdims=True)) + ROW * size
    dvar = ROW * var + 2 * dev * e + e * e
    rel = 0.55 * dvar / (var + eps) + 4 * U
    y = d * rstd * w + (0 if b is None else np.asarray(b, dtype=np.float64))
    size_y = np.abs(d * rstd * w)
    dy = (es + dmean) * rstd * np.abs(w) * (1 + rel) + size_y * (rel + 3 * U) + U * np.abs(y) + 1e-300
    return y, mean[:, 0], rstd[:, 0], dy, dmean[:, 0] + 1e-300, rel[:, 0]


def layernorm_backward(dy, h, w, mean, rstd, dh=None):
    """dx, dweight, dbias and bounds, from the stored h, mean and rstd."""
    dy, h, w = (np.asarray(t, dtype=np.float64) for t in (dy, h, w))
    mu, q = np.asarray(mean, dtype=np.float64)[:, None], np.asarray(rstd, dtype=np.float64)[:, None]
    xh, g = (h - mu) * q, dy * w
    avg = lambda t: np.mean(t, axis=1, keepdims=True)  # noqa: E731
    dx = q * (g - avg(g) - xh * avg(g * xh))
    bound = ROW * q * (np.abs(g) + avg(np.abs(g)) + np.abs(xh) * avg(np.abs(g * xh)))
    if dh is not None:
        dx = dx + np.asarray(dh, dtype=np.float64)
        bound = bound + 2 * U * np.abs(dh)
    return (dx, (dy * xh).sum(0), dy.sum(0), bound + 1e-45, COL * np.abs(dy * xh).sum(0) + 1e-45,
            COL * np.abs(dy).sum(0) + 1e-45)


def gated(z, dz, name):
    """h = act(gate) up for z = [gate, up] known to dz, and its bound."""
    I = z.shape[1] // 2
    g, u = z[:, :I], z[:, I:]
    eg, eu = (dz[:, :I], dz[:, I:]) if np.ndim(dz) else (dz, dz)
    a = ops.act(g, name)
    da = ops.act_bound(g, eg, name)
    return a * u, (np.abs(u) + eu) * da + np.abs(a) * eu + 2 * U * np.abs(a * u) + 1e-300


def gated_backward(dh, z, name):
    """p = [dh up act'(gate), dh act(gate)] and its bound."""
    I = z.shape[1] // 2
    g, u = z[:, :I], z[:, I:]
    a, s = ops.act(g, name), ops.act_slope(g, name)
    p = np.concatenate([dh * u * s, dh * a], 1)
    e = np.concatenate([np.abs(dh * u) * ops.slope_bound(g, name), np.abs(dh) * ops.act_bound(g, 0.0, name)], 1)
    return p, e + 4 * U * np.abs(p) + 1e-300


def check_fp8(y, dy, codes, sf, what):
    """codes (uint8 [n][I]) and scales (fp32 [n][I/128]) of values known to be within dy of y.
    A block's scale lies between those of its largest magnitude's two ends (an end of zero allows
    every smaller scale and 1, a block of zeros'); a code decodes to within dy plus half a code
    spacing; where both ends of a value round to one code under the only possible scale, the code
    is that one."""
    import oracle
    from tests.test_gpu_swiglu import E4M3, half_ulp_e4m3, oracle_nearest_mag
    n, I = y.shape
    yb, db = np.abs(y).reshape(n, I // 128, 128), dy.reshape(n, I // 128, 128)
    m, x = np.frexp(sf.astype(np.float64))
    assert np.all(m == 0.5), f"{what}: a scale is not a power of two"
    e = x - 1
    exp_of = np.vectorize(oracle.scale_exponent)
    low = np.max(np.maximum(yb - db, 0.0), axis=2)
    e_lo, e_hi = np.where(low > 0, exp_of(low), -10000), exp_of(np.max(yb + db, axis=2))
    ok = ((e >= e_lo) & (e <= e_hi)) | ((low == 0) & (e == 0))
    assert np.all(ok), f"{what}: {np.sum(~ok)} block scales outside the allowed range"
    s = np.repeat(np.ldexp(1.0, e), 128, axis=1)
    q = E4M3[codes].astype(np.float64) * s
    assert not np.any(np.isnan(q)), f"{what}: NaN code"
    slack = dy + half_ulp_e4m3((np.abs(y) + dy) / s) * s
    worst = np.max(np.abs(q - y) / slack)
    assert worst <= 1.0 + 1e-9, f"{what}: |decoded - y| reaches {worst:.3f} of the bound"
    lo, hi = (np.abs(y) - dy) / s, (np.abs(y) + dy) / s
    one = (lo > 0) & np.repeat(e_lo == e_hi, 128, axis=1)
    one &= oracle_nearest_mag(np.maximum(lo, 0)) == oracle_nearest_mag(hi)
    want = oracle_nearest_mag(np.abs(y) / s) | np.where(np.signbit(y), 0x80, 0)
    assert np.all(codes[one] == want[one]), f"{what}: {np.sum((codes != want) & one)} unambiguous codes differ"
