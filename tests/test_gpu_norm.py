"""GPU: the RMS norm with FP8 output (dg_rmsnorm_fp8_1x128), its backward
(dg_rmsnorm_backward) and the epilogue's backward (dg_bias_act_backward_fp8) against their
definitions in 64 bits (tests/_ops64.py, which also derives the bounds).

FP8 outputs: the interval check of the fused SwiGLU tests (scales between those that the
bound allows, codes within the bound plus half a code spacing, the oracle quantizer's code
wherever the interval leaves one choice). Outputs lie between seeded guard bands. h is exact.
"""
import numpy as np
import pytest
import torch

import oracle
from tests import _ops64 as ops
from tests import gpu_util as gu
from tests.test_gpu_quant import GuardedBytes
from tests.test_gpu_swiglu import check

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
EPS = 1e-6


def dg():
    import fp8_block_scaled_dg_amd as m
    return m


def hidden(seed, M, K, dtype):
    """Normal rows of sizes from 2^-6 to 2^6, a few channels twelve times larger."""
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(M, K, generator=g) * torch.where(torch.rand(K, generator=g) < 0.01, 12.0, 1.0)
    return (x * 2.0 ** torch.randint(-6, 7, (M, 1), generator=g)).to(dtype)


def weights(seed, K, dtype):
    g = torch.Generator().manual_seed(seed)
    return (1 + 0.3 * torch.randn(K, generator=g)).to(dtype)


def scale_values(sf, KB):
    """fp32 scales from either form; the packed form's padding bytes have to be zero."""
    if sf.dtype == F32:
        return sf.cpu().numpy()
    b = sf.view(torch.uint8).cpu().numpy()
    assert not b[:, KB:].any(), "padding bytes of the packed scales"
    return np.ldexp(1.0, b[:, :KB].astype(np.int32) - 127).astype(np.float32)


class Fp8Out:
    """Guarded codes [M, K] and scales of either form."""

    def __init__(self, M, K, packed, seed=3):
        KB = K // 128
        self.M, self.K, self.KB = M, K, KB
        width = (KB + 3) // 4 if packed else KB
        self._c, self._s = GuardedBytes(M * K, seed), GuardedBytes(M * width * 4, seed + 1)
        self.codes = self._c.view(torch.float8_e4m3fn, (M, K))
        self.sf = self._s.view(torch.int32 if packed else F32, (M, width))

    def result(self):
        torch.cuda.synchronize()
        assert self._c.guards_intact() and self._s.guards_intact(), "write outside the outputs"
        return self._c.result().reshape(self.M, self.K), scale_values(self.sf, self.KB)


def run_norm(x, r, w, packed=False, h=None, eps=EPS, rstd=True):
    M, K = x.shape
    out = Fp8Out(M, K, packed)
    rs = torch.full((M,), -7.0, device="cuda") if rstd else None
    gu.announce(f"rmsnorm {x.dtype} M={M} K={K} residual={r is not None} packed={packed}")
    dg().rmsnorm_fp8_1x128(x, w, eps, residual=r, h=h, rstd=rs, codes=out.codes, sf=out.sf)
    codes, sf = out.result()
    return codes, sf, rs.cpu().numpy() if rstd else None


def check_norm(x, r, w, codes, sf, rstd, what, eps=EPS):
    y, _, q = ops.rmsnorm(x.double().numpy(), None if r is None else r.double().numpy(),
                          w.double().numpy(), eps)
    assert np.max(np.abs(rstd / q - 1)) <= ops.RSTD_REL, what
    check(y, np.abs(y) * ops.Y_REL + 1e-300, codes, sf, what, strict=True)


@pytest.mark.parametrize("M,K", [(1, 128), (1, 7168), (3, 384), (5, 1024), (7, 1152), (257, 2048),
                                 (64, 7168), (2, 16384), (3, 16512), (2, 18432), (2, 32768), (5000, 256)])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_norm(M, K, dtype):
    x, r = hidden(M + K, M, K, dtype), hidden(M + K + 1, M, K, dtype)
    for res, wt, packed in ((False, BF, False), (True, F32, True)):
        w = weights(K, K, wt)
        rr = r if res else None
        h = torch.zeros(M, K, dtype=dtype, device="cuda") if res else None
        codes, sf, rstd = run_norm(x.cuda(), None if rr is None else rr.cuda(), w.cuda(), packed, h)
        check_norm(x, rr, w, codes, sf, rstd, f"{dtype} {M}x{K} residual={res}")
        if res:  # the fp32 sum, rounded once: no freedom
            assert torch.equal(h.cpu(), (x.float() + r.float()).to(dtype))


def test_norm_scale_forms_and_optional_outputs_agree():
    x, r, w = hidden(1, 33, 1152, BF).cuda(), hidden(2, 33, 1152, BF).cuda(), weights(3, 1152, BF).cuda()
    c0, s0, _ = run_norm(x, r, w, packed=False)
    c1, s1, _ = run_norm(x, r, w, packed=True, rstd=False)
    assert np.array_equal(c0, c1) and np.array_equal(s0, s1)
    c2, s2 = dg().rmsnorm_fp8_1x128(x, w, EPS, residual=r, ue8m0=True)
    assert np.array_equal(c2.view(torch.uint8).cpu().numpy(), c0)
    assert np.array_equal(scale_values(s2, 9), s0)


@pytest.mark.parametrize("which", ["x", "residual"])
def test_norm_in_place_sum(which):
    x, r, w = hidden(4, 600, 2048, BF).cuda(), hidden(5, 600, 2048, BF).cuda(), weights(6, 2048, BF).cuda()
    want = run_norm(x, r, w)
    total = (x.float() + r.float()).to(BF)
    a, b = x.clone(), r.clone()
    got = run_norm(a, b, w, h=a if which == "x" else b)
    assert np.array_equal(got[0], want[0]) and np.array_equal(got[1], want[1])
    assert torch.equal(a if which == "x" else b, total)
    assert torch.equal(b if which == "x" else a, r if which == "x" else x)


def test_norm_special_rows():
    K = 512
    x = torch.zeros(8, K)
    x[1] = -0.0
    x[2] = torch.linspace(-1, 1, K) * 1e-25          # squares underflow: eps alone counts
    x[3, 7], x[4, 200], x[5, 300] = float("nan"), float("inf"), float("-inf")
    x[6] = 3e30                                       # squares overflow
    x[7, 100] = 5.0                                   # one value carries the row
    codes, sf, rstd = run_norm(x.cuda(), None, torch.ones(K).cuda())
    assert not (codes[0] & 0x7F).any() and np.all(codes[1] == 0x80) and np.all(sf[:2] == 1)
    assert np.allclose(rstd[:3], 1e3, rtol=2.0 ** -20)
    y = ops.rmsnorm(x[2:3].numpy(), None, np.ones(K), EPS)[0]
    check(y, np.abs(y) * ops.Y_REL, codes[2:3], sf[2:3], "tiny row", strict=True)
    assert np.all((codes[3] & 0x7F) == 0x7F) and np.isnan(rstd[3])
    for row, at in ((4, 200), (5, 300)):              # inf * 0 at the infinity, zero elsewhere
        assert rstd[row] == 0 and (codes[row, at] & 0x7F) == 0x7F
        assert not (np.delete(codes[row], at) & 0x7F).any()
    assert rstd[6] == 0 and not (codes[6] & 0x7F).any()
    assert np.count_nonzero(codes[7] & 0x7F) == 1


def test_norm_packed_scale_floor():
    # y of 2^-139: the packed form's least exponent is -127, the codes go to zero
    x = torch.full((1, 128), 2.0 ** -120)
    w = torch.full((128,), 2.0 ** -29)
    codes, sf, _ = run_norm(x.cuda(), None, w.cuda(), packed=True)
    assert sf[0, 0] == np.float32(2.0 ** -127) and not (codes & 0x7F).any()


def test_norm_and_gradients_on_another_stream_and_repeated():
    x, r, w = hidden(7, 300, 4096, BF).cuda(), hidden(8, 300, 4096, BF).cuda(), weights(9, 4096, BF).cuda()
    dy = hidden(10, 300, 4096, BF).cuda()

    def everything():
        h, rstd = torch.empty_like(x), torch.empty(300, device="cuda")
        codes, sf = dg().rmsnorm_fp8_1x128(x, w, EPS, residual=r, h=h, rstd=rstd)
        dx, dw = dg().rmsnorm_backward(dy, h, w, rstd, dh=r)
        ac, asf, db = dg().bias_act_backward_fp8(dy, x, "gelu")
        return [codes.view(torch.uint8), sf, h, rstd, dx, dw, ac.view(torch.uint8), asf, db]

    want = everything()
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        got = everything()
    again = everything()
    torch.cuda.synchronize()
    for a, b, c in zip(want, got, again):
        assert torch.equal(a, b) and torch.equal(a, c)


def test_norm_rows_past_32_bit_offsets():
    # 2^32 values and more: the last rows equal those of a small call
    K = 8192
    M = (1 << 32) // K + 3
    x = torch.empty(M, K, dtype=BF, device="cuda")
    base = hidden(11, 64, K, BF).cuda()
    x.view(-1)[: (M // 64) * 64 * K].view(-1, 64, K).copy_(base.expand(M // 64, 64, K))
    x[(M // 64) * 64:] = base[: M % 64].flip(0)
    w = weights(12, K, BF).cuda()
    gu.announce(f"rmsnorm M={M} K={K}")
    codes, sf = dg().rmsnorm_fp8_1x128(x, w, EPS)
    c0, s0 = dg().rmsnorm_fp8_1x128(x[-5:].contiguous(), w, EPS)
    torch.cuda.synchronize()
    assert torch.equal(codes[-5:].view(torch.uint8), c0.view(torch.uint8)) and torch.equal(sf[-5:], s0)
    del codes, sf
    gu.announce(f"act backward M={M} N={K}")
    dc, dsf, _ = dg().bias_act_backward_fp8(x, None, None, need_dbias=False)
    d0, ds0, _ = dg().bias_act_backward_fp8(x[-5:].contiguous(), None, None, need_dbias=False)
    torch.cuda.synchronize()
    assert torch.equal(dc[-5:].view(torch.uint8), d0.view(torch.uint8)) and torch.equal(dsf[-5:], ds0)
    del dc, dsf
    gu.announce(f"rmsnorm backward M={M} K={K}")
    rstd = torch.rand(M, device="cuda")
    dx, _ = dg().rmsnorm_backward(x, x, w, rstd)
    dx0, _ = dg().rmsnorm_backward(x[-5:].contiguous(), x[-5:].contiguous(), w, rstd[-5:].contiguous())
    torch.cuda.synchronize()
    assert torch.equal(dx[-5:], dx0)


# ---------------------------------------------------------------- backward of the norm

@pytest.mark.parametrize("M,K", [(1, 128), (1, 7168), (3, 384), (7, 1152), (257, 2048), (64, 7168),
                                 (3, 16512), (5, 18432), (2, 32768), (3000, 256), (300, 16512), (256, 1024),
                                 (600, 9216)])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_norm_backward(M, K, dtype):
    h, dy, dh = (hidden(100 * s + M + K, M, K, dtype) for s in range(3))
    for res, wt in ((False, BF), (True, F32)):
        w = weights(K, K, wt)
        rstd = torch.rsqrt(h.double().square().mean(1) + EPS).float()
        dx = gu.Guarded((M, K * (2 if dtype == F32 else 1)), 17)
        dw = torch.full((K + 8,), 5.0, device="cuda")
        gu.announce(f"rmsnorm backward {dtype} M={M} K={K} dh={res}")
        dg().rmsnorm_backward(dy.cuda(), h.cuda(), w.cuda(), rstd.cuda(), dh=dh.cuda() if res else None,
                              dx=dx.out.view(dtype).view(M, K), dweight=dw[4:K + 4])
        torch.cuda.synchronize()
        assert dx.guards_intact() and torch.all(dw[:4] == 5) and torch.all(dw[-4:] == 5)
        want, wantw, bx, bw = ops.rmsnorm_backward(dy.double().numpy(), h.double().numpy(), w.double().numpy(),
                                                   rstd.double().numpy(), dh.double().numpy() if res else None)
        got = dx.out.view(dtype).view(M, K).double().cpu().numpy()
        own = ops.bf16_slack(np.abs(want) + bx) if dtype == BF else 2 * ops.U * np.abs(want) + 1e-45
        assert np.all(np.abs(got - want) <= bx + own), f"dx {M}x{K}"
        err = np.abs(dw[4:K + 4].double().cpu().numpy() - wantw)
        assert np.all(err <= bw + 1e-45), f"dweight {M}x{K}: {np.max(err / (bw + 1e-45))}"


@pytest.mark.parametrize("which", ["dy", "dh", "h"])
def test_norm_backward_in_place(which):
    h, dy, dh = (hidden(s, 700, 2048, BF).cuda() for s in (21, 22, 23))
    w, rstd = weights(24, 2048, BF).cuda(), torch.rand(700, device="cuda")
    want, wantw = dg().rmsnorm_backward(dy, h, w, rstd, dh=dh)
    t = dict(dy=dy.clone(), h=h.clone(), dh=dh.clone())
    got, gotw = dg().rmsnorm_backward(t["dy"], t["h"], w, rstd, dh=t["dh"], dx=t[which])
    torch.cuda.synchronize()
    assert torch.equal(got, want) and torch.equal(gotw, wantw)


@pytest.mark.parametrize("M,K", [(1, 7168), (64, 512), (200, 7168), (256, 16512)])
@pytest.mark.parametrize("which", ["dy", "dh", "h"])
def test_norm_backward_in_place_of_few_rows(M, K, which):
    # the sums of few rows read the inputs again: dx must not overwrite them before
    h, dy, dh = (hidden(s, M, K, F32) for s in (25, 26, 27))
    w, rstd = weights(28, K, F32), torch.rand(M)
    want, _ = dg().rmsnorm_backward(dy.cuda(), h.cuda(), w.cuda(), rstd.cuda(), dh=dh.cuda())
    t = dict(dy=dy.cuda(), h=h.cuda(), dh=dh.cuda())
    got, gotw = dg().rmsnorm_backward(t["dy"], t["h"], w.cuda(), rstd.cuda(), dh=t["dh"], dx=t[which])
    torch.cuda.synchronize()
    _, wantw, _, bw = ops.rmsnorm_backward(dy.double().numpy(), h.double().numpy(), w.double().numpy(),
                                           rstd.double().numpy(), dh.double().numpy())
    assert torch.equal(got, want)
    assert np.all(np.abs(gotw.double().cpu().numpy() - wantw) <= bw + 1e-45)


def test_norm_backward_is_the_difference_quotient_of_the_forward_norm():
    # directional difference of sum(dy * y) on the fp64 formula with the forward's own rstd
    M, K = 40, 1024
    h, w, dy = hidden(31, M, K, F32), weights(32, K, F32), hidden(33, M, K, F32)
    rstd = torch.empty(M, device="cuda")
    dg().rmsnorm_fp8_1x128(h.cuda(), w.cuda(), EPS, rstd=rstd)
    dx, dw = (t.double().cpu().numpy() for t in dg().rmsnorm_backward(dy.cuda(), h.cuda(), w.cuda(), rstd))
    h, w, dy = h.double().numpy(), w.double().numpy(), dy.double().numpy()
    rng = np.random.default_rng(34)
    size = np.sqrt(np.mean(h * h, axis=1, keepdims=True))
    for _ in range(8):
        d, e, t = rng.normal(size=(M, K)) * size, rng.normal(size=K), 1e-5
        loss = lambda s: float((ops.rmsnorm(h + s * d, None, w + s * e, EPS)[0] * dy).sum())  # noqa: E731
        slope = (loss(t) - loss(-t)) / (2 * t)
        scale = np.abs(dx * d).sum() + np.abs(dw * e).sum()
        assert abs(slope - (dx * d).sum() - (dw * e).sum()) <= 2.0 ** -16 * scale


def test_backward_of_no_rows_writes_zeros():
    e = torch.zeros(0, 256, dtype=BF, device="cuda")
    dx, dw = dg().rmsnorm_backward(e, e, torch.ones(256, device="cuda"), torch.zeros(0, device="cuda"),
                                   dweight=torch.full((256,), 9.0, device="cuda"))
    codes, sf, db = dg().bias_act_backward_fp8(e, e, "relu", dbias=torch.full((256,), 9.0, device="cuda"))
    c2, s2 = dg().rmsnorm_fp8_1x128(e, torch.ones(256, device="cuda"))
    torch.cuda.synchronize()
    assert dx.shape == codes.shape == c2.shape == (0, 256) and not dw.any() and not db.any()


# ---------------------------------------------------------------- backward of the epilogue

@pytest.mark.parametrize("M,N", [(1, 128), (1, 18432), (3, 384), (5, 1024), (130, 2048), (257, 1152),
                                 (4100, 256), (64, 7168), (130, 12288)])
@pytest.mark.parametrize("act", ops.ACTS)
def test_act_backward(M, N, act):
    g = torch.Generator().manual_seed(M + N)
    dc = hidden(M * N, M, N, BF)
    pre = (2.5 * torch.randn(M, N, generator=g)).to(BF)
    pre.view(-1)[::97] = 0.0
    packed = act in ("silu", "none")
    out = Fp8Out(M, N, packed)
    db = torch.full((N + 8,), 5.0, device="cuda")
    gu.announce(f"act backward {act} M={M} N={N}")
    dg().bias_act_backward_fp8(dc.cuda(), None if act == "none" else pre.cuda(), act, codes=out.codes,
                               sf=out.sf, dbias=db[4:N + 4])
    codes, sf = out.result()
    assert torch.all(db[:4] == 5) and torch.all(db[-4:] == 5)
    d, z = dc.double().numpy(), pre.double().numpy()
    p = d * ops.act_slope(z, act)
    dp = np.abs(d) * ops.slope_bound(z, act) + 2 * ops.U * np.abs(p) + 1e-300
    if act in ("none", "relu"):  # p is exact: the oracle quantizer's bytes
        rc, rs = oracle.quantize_blocks(p.astype(np.float32), 1, 128)
        assert np.array_equal(rs, sf) and np.array_equal(rc & 0x7F, codes & 0x7F)
        assert np.array_equal(rc[p != 0], codes[p != 0])
    else:
        check(p, dp, codes, sf, f"{act} {M}x{N}", strict=False)
    # dbias: sums at most 200 values and partials deep
    err = np.abs(db[4:N + 4].double().cpu().numpy() - p.sum(0))
    assert np.all(err <= 2.0 ** -16 * np.abs(p).sum(0) + dp.sum(0) + 1e-45), f"{act} dbias"


def test_act_backward_without_dbias_and_forms_agree():
    dc, pre = hidden(41, 70, 1152, BF).cuda(), hidden(42, 70, 1152, BF).cuda()
    c0, s0, db = dg().bias_act_backward_fp8(dc, pre, "silu")
    c1, s1, none = dg().bias_act_backward_fp8(dc, pre, "silu", need_dbias=False, ue8m0=True)
    torch.cuda.synchronize()
    assert none is None and db.shape == (1152,)
    assert torch.equal(c0.view(torch.uint8), c1.view(torch.uint8))
    assert np.array_equal(s0.cpu().numpy(), scale_values(s1, 9))


def test_act_backward_agrees_with_the_quantizer():
    x = hidden(43, 77, 1024, BF).cuda()
    want = dg().quantize_fp8_1x128(x)
    got = dg().bias_act_backward_fp8(x, need_dbias=False)
    torch.cuda.synchronize()
    assert torch.equal(got[0].view(torch.uint8), want[0].view(torch.uint8)) and torch.equal(got[1], want[1])
