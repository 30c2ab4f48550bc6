"""GPU: the slopes of the epilogue's activations (dg_bias_act_backward_fp8) at every finite
bf16 pre-activation, tails and largest values included, against their definitions in 64 bits.

With one row of nonzero dc, dbias is the row's own dc * act'(pre) in fp32, so that each slope
is held to the roundings of its own formula (act_slope_bounds) and not to a flat bound that a
tail of 1e-20 would pass with any value. One row takes the call's one-launch form, 257 rows
the form with partial sums; the other rows' zeros also show a slope that is not finite."""
import numpy as np
import pytest
import torch
from scipy.special import erfcx, expit

from tests import _ops64 as ops
from tests import gpu_util as gu
from tests.test_gpu_norm import BF, Fp8Out, dg
from tests.test_gpu_swiglu import check

pytestmark = pytest.mark.gpu
U = ops.U


def act_slope_bounds(z, name):
    """|act' in fp32 - act'(z)|, z exact, counting roundings (U relative each).

    sigmoid(v): exp2 of -v log2 e: the argument's roundings give 2 |v| U, exp2 and the
    reciprocal 2 U each, the sum 1: with w = the relative error of v in units of U,
    rel(s) <= (5 + (2 + w) |v|) U. 1 - s: 4 U and s (1 - s) of the power's error, or exactly
    0 where 1 + e^-v rounds to 1. A power below 2^-126 counts as zero: 2^-115 covers it
    with the factors of up to 2^9 that it meets."""
    a = np.abs(z)
    if name in ("none", "relu"):
        return np.zeros_like(z)
    if name == "gelu":
        # (tail - phi0 a) bell: the polynomial and its steps 16 U, e^(-a^2/2) 2 U and 2 a^2 U
        tail, bell = 0.5 * erfcx(a / np.sqrt(2)), np.exp(-a * a / 2)
        rel = (20 + 2 * np.minimum(a * a, 1e4)) * U
        return (tail + 0.4 * a) * bell * rel + np.where(z > 0, 2 * U, 0.0) + 2.0 ** -115
    if name == "silu":
        v, dv, w = z, np.ones_like(z), 0
    else:  # gelu_tanh: v = 2u by four roundings, du/dx likewise
        v = 2 * ops.C_TANH * (z + 0.044715 * z ** 3)
        dv, w = 2 * ops.C_TANH * (1 + 3 * 0.044715 * z * z), 4
    s, c = expit(v), expit(-v)
    av = np.minimum(np.abs(v), 1e4)  # beyond, s and 1 - s are 0 or 1
    rel = (5 + (2 + w) * av) * U
    d1 = np.where(c < U / 4, c, 4 * U + s * c * (2 + (2 + w) * av) * U)
    term = np.where(s * c > 0, a * s * c * dv, 0.0)
    one = np.where(s * d1 > 0, a * s * d1 * dv, 0.0)
    return s * rel + term * (rel + 8 * U) + one + 2.0 ** -115


def finite_bf16():
    """Every finite bf16 value, a binade of one sign per 128: [65280]."""
    bits = np.arange(65536, dtype=np.uint32) << 16
    v = bits.astype(np.uint32).view(np.float32)
    return v[np.isfinite(v)]


@pytest.mark.parametrize("M", [1, 257])
@pytest.mark.parametrize("act", ops.ACTS)
def test_slopes_at_every_finite_value(act, M):
    z = finite_bf16()
    N = z.size
    g = torch.Generator().manual_seed(M)
    pre = torch.from_numpy(z)[None, :].repeat(M, 1)
    pre[1:] = pre[1:].roll(64, 1)  # other values under the zeros
    dc = torch.zeros(M, N)
    dc[0] = torch.randn(N, generator=g).sign() * (1 + torch.rand(N, generator=g))
    dc, pre = dc.to(BF), pre.to(BF)
    out = Fp8Out(M, N, False)
    db = torch.full((N,), 5.0, device="cuda")
    gu.announce(f"act slopes {act} M={M} N={N}")
    dg().bias_act_backward_fp8(dc.cuda(), pre.cuda(), act, codes=out.codes, sf=out.sf, dbias=db)
    codes, sf = out.result()
    d, x = dc[0].double().numpy(), z.astype(np.float64)
    p = d * ops.act_slope(x, act)
    dp = np.abs(d) * act_slope_bounds(x, act) + U * np.abs(p)
    got = db.double().cpu().numpy()
    bad = ~(np.abs(got - p) <= dp)
    assert not bad.any(), f"{act}: {bad.sum()} slopes, first at {x[bad][:4]}: {got[bad][:4]}, not {p[bad][:4]}"
    assert not (codes[1:] & 0x7F).any(), "dc of zero"
    # blocks that are not below what fp32 holds
    seen = np.abs(p).reshape(-1, 128).max(1) > 4 * dp.reshape(-1, 128).max(1)
    block = lambda t: t.reshape(-1, 128)[seen].reshape(1, -1)  # noqa: E731
    check(block(p), block(dp), block(codes[0]), sf[0][seen][None, :], f"{act} M={M}", strict=False)
