"""GPU: the layer norm of residual + dropout(x) with FP8 output (dg_layernorm_fp8_1x128) and its
backward (dg_layernorm_backward) against their definitions in 64 bits (tests/_block64.py, which
also derives the bounds). FP8 outputs: the interval check of _block64. Outputs lie
between seeded guard bands."""
import numpy as np
import pytest
import torch

from tests import _block64 as blk
from tests import _ops64 as ops
from tests import gpu_util as gu
from tests.test_gpu_dropout import OFFSET, SEED, rng_state
from tests.test_gpu_norm import BF, F32, Fp8Out, hidden, weights

pytestmark = pytest.mark.gpu
EPS = 1e-5


def dg():
    import fp8_block_scaled_dg_amd as m
    return m


def off_center(seed, M, K, dtype):
    """Rows of several sizes about means of several sizes."""
    g = torch.Generator().manual_seed(seed)
    mean = torch.randn(M, 1, generator=g) * 2.0 ** torch.randint(-4, 5, (M, 1), generator=g)
    return (hidden(seed, M, K, F32) + mean).to(dtype)


def run_norm(x, w, b=None, r=None, packed=False, h=None, stats=True, p=0.0, sub=0, eps=EPS):
    M, K = x.shape
    out = Fp8Out(M, K, packed)
    st = torch.full((2, M + 8), -7.0, device="cuda")
    mean, rstd = (st[0, 4:M + 4], st[1, 4:M + 4]) if stats else (None, None)
    gu.announce(f"layernorm {x.dtype} M={M} K={K} residual={r is not None} p={p} packed={packed}")
    dg().layernorm_fp8_1x128(x, w, b, eps, residual=r, h=h, mean=mean, rstd=rstd, codes=out.codes, sf=out.sf,
                             dropout_p=p, rng=rng_state() if p else None, subsequence=sub)
    codes, sf = out.result()
    assert torch.all(st[:, :4] == -7) and torch.all(st[:, -4:] == -7)
    return codes, sf, *((mean.cpu().numpy(), rstd.cpu().numpy()) if stats else (None, None))


def check_norm(x, w, b, r, got, what, p=0.0, sub=0, eps=EPS):
    codes, sf, mean, rstd = got
    s, es = blk.sum_before_norm(x.double().numpy(), None if r is None else r.double().numpy(), p, SEED, OFFSET, sub)
    y, m, q, dy, dm, rel = blk.layernorm(s, es, w.double().numpy(), None if b is None else b.double().numpy(), eps)
    assert np.all(np.abs(mean - m) <= dm), what
    assert np.all(np.abs(rstd / q - 1) <= rel), what
    blk.check_fp8(y, dy, codes, sf, what)
    return s, es


@pytest.mark.parametrize("M,K", [(1, 128), (1, 7168), (3, 384), (5, 1024), (7, 1152), (257, 2048), (64, 7168),
                                 (2, 16384), (3, 16512), (2, 18432), (2, 32768), (5000, 256), (300, 9216)])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_layernorm(M, K, dtype):
    x, r = off_center(M + K, M, K, dtype), off_center(M + K + 1, M, K, dtype)
    for res, wt, bias, packed, p in ((False, BF, False, False, 0.0), (True, F32, True, True, 0.0),
                                     (True, BF, True, False, 0.1), (False, F32, False, False, 0.5)):
        w, b = weights(K, K, wt), (weights(K + 1, K, wt) - 1).to(wt) if bias else None
        rr = r if res else None
        h = gu.Guarded((M, K * (2 if dtype == F32 else 1)), 9)
        got = run_norm(x.cuda(), w.cuda(), b.cuda() if bias else None, r.cuda() if res else None, packed,
                       h.out.view(dtype).view(M, K), p=p, sub=M)
        what = f"{dtype} {M}x{K} residual={res} p={p}"
        s, es = check_norm(x, w, b, rr, got, what, p, M)
        assert h.guards_intact()
        hv = h.out.view(dtype).view(M, K)
        if p == 0:  # the fp32 sum, rounded once: no freedom
            want = (x.float() + r.float()).to(dtype) if res else x
            assert torch.equal(hv.cpu(), want), what
        own = ops.bf16_slack(np.abs(s) + es) if dtype == BF else 0
        assert np.all(np.abs(hv.double().cpu().numpy() - s) <= es + own), what


def test_layernorm_dropout_is_dropout_add():
    # the sum before the norm equals what dropout_add gives, bit for bit
    for dtype in (BF, F32):
        x, r, w = off_center(1, 130, 2176, dtype).cuda(), off_center(2, 130, 2176, dtype).cuda(), weights(3, 2176, BF).cuda()
        h = torch.empty_like(x)
        run_norm(x, w, None, r, h=h, p=0.3, sub=77)
        want = dg().dropout_add(x, 0.3, rng_state(), 77, residual=r)
        torch.cuda.synchronize()
        assert torch.equal(h, want)


def test_layernorm_scale_forms_and_optional_outputs_agree():
    x, r, w = off_center(1, 33, 1152, BF).cuda(), off_center(2, 33, 1152, BF).cuda(), weights(3, 1152, BF).cuda()
    c0, s0, *_ = run_norm(x, w, w, r)
    c1, s1, *_ = run_norm(x, w, w, r, packed=True, stats=False)
    assert np.array_equal(c0, c1) and np.array_equal(s0, s1)
    c2, s2 = dg().layernorm_fp8_1x128(x, w, w, EPS, residual=r, ue8m0=True)
    assert np.array_equal(c2.view(torch.uint8).cpu().numpy(), c0) and s2.dtype == torch.int32


@pytest.mark.parametrize("which", ["x", "residual"])
def test_layernorm_in_place_sum(which):
    x, r, w = off_center(4, 600, 2048, BF).cuda(), off_center(5, 600, 2048, BF).cuda(), weights(6, 2048, BF).cuda()
    h = torch.empty_like(x)
    want = run_norm(x, w, None, r, h=h, p=0.1)
    a, b = x.clone(), r.clone()
    got = run_norm(a, w, None, b, h=a if which == "x" else b, p=0.1)
    assert all(np.array_equal(g, t) for g, t in zip(got, want))
    assert torch.equal(a if which == "x" else b, h) and torch.equal(b if which == "x" else a, r if which == "x" else x)


def test_layernorm_far_mean():
    # mean 1000 deviations away: a difference of two sums would leave no digits of the variance
    x = 4096 + torch.randn(40, 4096, generator=torch.Generator().manual_seed(8))
    w = torch.ones(4096)
    check_norm(x, w, None, None, run_norm(x.cuda(), w.cuda()), "far mean")
    x = torch.full((3, 1024), 3.25)  # no variance at all
    codes, _, mean, rstd = run_norm(x.cuda(), torch.ones(1024).cuda())
    assert np.all(mean == 3.25) and np.allclose(rstd, EPS ** -0.5, rtol=2.0 ** -20) and not (codes & 0x7F).any()


def test_layernorm_special_rows():
    K = 512
    x = torch.zeros(7, K)
    x[1] = -0.0
    x[2] = torch.linspace(-1, 1, K) * 1e-25           # squares underflow: eps alone counts
    x[3, 7], x[4, 200], x[5, 300] = float("nan"), float("inf"), float("-inf")
    x[6] = torch.where(torch.arange(K) % 2 == 0, 3e30, -3e30)  # squares overflow
    codes, sf, mean, rstd = run_norm(x.cuda(), torch.ones(K).cuda())
    assert not (codes[:2] & 0x7F).any() and np.all(sf[:2] == 1)
    assert np.allclose(rstd[:3], EPS ** -0.5, rtol=2.0 ** -20)
    for row in (3, 4, 5):                              # the mean is not finite, no difference from it is
        assert np.all((codes[row] & 0x7F) == 0x7F) and np.isnan(rstd[row]) and not np.isfinite(mean[row])
    assert rstd[6] == 0 and not (codes[6] & 0x7F).any()
    # the rows beside them are what they are alone
    alone = run_norm(x[2:3].cuda(), torch.ones(K).cuda())
    assert np.array_equal(alone[0], codes[2:3]) and np.array_equal(alone[1], sf[2:3])


def test_layernorm_rows_past_32_bit_offsets():
    K = 8192
    M = (1 << 32) // K + 3
    x = torch.empty(M, K, dtype=BF, device="cuda")
    base = off_center(11, 64, K, BF).cuda()
    x.view(-1)[: (M // 64) * 64 * K].view(-1, 64, K).copy_(base.expand(M // 64, 64, K))
    x[(M // 64) * 64:] = base[: M % 64].flip(0)
    w = weights(12, K, BF).cuda()
    gu.announce(f"layernorm M={M} K={K}")
    codes, sf = dg().layernorm_fp8_1x128(x, w)
    c0, s0 = dg().layernorm_fp8_1x128(x[-5:].contiguous(), w)
    torch.cuda.synchronize()
    assert torch.equal(codes[-5:].view(torch.uint8), c0.view(torch.uint8)) and torch.equal(sf[-5:], s0)
    gu.announce(f"layernorm with dropout M={M} K={K}")
    rows = torch.ones(1, K, device="cuda")
    h = torch.empty_like(x)
    dg().layernorm_fp8_1x128(x, w, h=h, dropout_p=0.5, rng=rng_state(), codes=codes, sf=sf)
    torch.cuda.synchronize()
    keep = blk.kept((M - 1) * K, K, 0.5, SEED, OFFSET)
    assert np.array_equal((h[-1] != 0).cpu().numpy(), keep & (x[-1] != 0).cpu().numpy()) and rows.any()
    del codes, sf, h
    gu.announce(f"layernorm backward M={M} K={K}")
    mean, rstd = torch.randn(M, device="cuda"), torch.rand(M, device="cuda")
    dx, *_ = dg().layernorm_backward(x, x, w, mean, rstd)
    t = x[-5:].contiguous()
    dx0, *_ = dg().layernorm_backward(t, t, w, mean[-5:].contiguous(), rstd[-5:].contiguous())
    torch.cuda.synchronize()
    assert torch.equal(dx[-5:], dx0)


# ---------------------------------------------------------------- backward

@pytest.mark.parametrize("M,K", [(1, 128), (1, 7168), (3, 384), (7, 1152), (257, 2048), (64, 7168), (3, 16512),
                                 (5, 18432), (2, 32768), (3000, 256), (300, 16512), (256, 1024), (600, 9216),
                                 (270, 32768), (2100, 128)])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_layernorm_backward(M, K, dtype):
    h = off_center(M + K, M, K, dtype)
    dy, dh = (hidden(100 * s + M + K, M, K, dtype) for s in (1, 2))
    mean = h.double().mean(1)
    rstd = torch.rsqrt((h.double() - mean[:, None]).square().mean(1) + EPS).float()
    mean = mean.float()
    for res, wt in ((False, BF), (True, F32)):
        w = weights(K, K, wt)
        dx = gu.Guarded((M, K * (2 if dtype == F32 else 1)), 17)
        sums = torch.full((2, K + 8), 5.0, device="cuda")
        gu.announce(f"layernorm backward {dtype} M={M} K={K} dh={res}")
        dg().layernorm_backward(dy.cuda(), h.cuda(), w.cuda(), mean.cuda(), rstd.cuda(), dh=dh.cuda() if res else None,
                                dx=dx.out.view(dtype).view(M, K), dweight=sums[0, 4:K + 4], dbias=sums[1, 4:K + 4])
        torch.cuda.synchronize()
        assert dx.guards_intact() and torch.all(sums[:, :4] == 5) and torch.all(sums[:, -4:] == 5)
        wx, ww, wb, bx, bw, bb = blk.layernorm_backward(
            dy.double().numpy(), h.double().numpy(), w.double().numpy(), mean.double().numpy(),
            rstd.double().numpy(), dh.double().numpy() if res else None)
        got = dx.out.view(dtype).view(M, K).double().cpu().numpy()
        own = ops.bf16_slack(np.abs(wx) + bx) if dtype == BF else 2 * ops.U * np.abs(wx)
        assert np.all(np.abs(got - wx) <= bx + own), f"dx {M}x{K}"
        gw, gb = (t[4:K + 4].double().cpu().numpy() for t in sums)
        assert np.all(np.abs(gw - ww) <= bw), f"dweight {M}x{K}"
        assert np.all(np.abs(gb - wb) <= bb), f"dbias {M}x{K}"


@pytest.mark.parametrize("M,K", [(1, 7168), (64, 512), (200, 7168), (256, 16512), (700, 2048), (300, 128)])
@pytest.mark.parametrize("which", ["dy", "dh", "h"])
def test_layernorm_backward_in_place(M, K, which):
    # the sums of few rows read the inputs again: dx must not overwrite them before
    h, dy, dh = (off_center(s, M, K, F32) for s in (25, 26, 27))
    w, mean, rstd = weights(28, K, F32), torch.randn(M), torch.rand(M)
    args = w.cuda(), mean.cuda(), rstd.cuda()
    want, ww, wb = dg().layernorm_backward(dy.cuda(), h.cuda(), *args, dh=dh.cuda())
    t = dict(dy=dy.cuda(), h=h.cuda(), dh=dh.cuda())
    got, gw, gb = dg().layernorm_backward(t["dy"], t["h"], *args, dh=t["dh"], dx=t[which])
    _, w2, none = dg().layernorm_backward(dy.cuda(), h.cuda(), *args, dh=dh.cuda(), need_dbias=False)
    torch.cuda.synchronize()
    _, ew, eb, _, bw, bb = blk.layernorm_backward(dy.double().numpy(), h.double().numpy(), w.double().numpy(),
                                                  mean.double().numpy(), rstd.double().numpy(), dh.double().numpy())
    assert torch.equal(got, want) and none is None and torch.equal(w2, ww)
    assert np.all(np.abs(gw.double().cpu().numpy() - ew) <= bw) and np.all(np.abs(gb.double().cpu().numpy() - eb) <= bb)
    assert np.all(np.abs(wb.double().cpu().numpy() - eb) <= bb)


def test_layernorm_backward_is_the_difference_quotient_of_the_forward_norm():
    # directional difference of sum(dy * y) on the fp64 formula with the forward's own statistics
    M, K = 40, 1024
    h, w, b, dy = off_center(31, M, K, F32), weights(32, K, F32), weights(33, K, F32), hidden(34, M, K, F32)
    mean, rstd = torch.empty(M, device="cuda"), torch.empty(M, device="cuda")
    dg().layernorm_fp8_1x128(h.cuda(), w.cuda(), b.cuda(), EPS, mean=mean, rstd=rstd)
    dx, dw, db = (t.double().cpu().numpy() for t in dg().layernorm_backward(dy.cuda(), h.cuda(), w.cuda(), mean, rstd))
    h, w, b, dy = (t.double().numpy() for t in (h, w, b, dy))
    rng = np.random.default_rng(35)
    size = h.std(1, keepdims=True)
    for _ in range(8):
        d, e, f, t = rng.normal(size=(M, K)) * size, rng.normal(size=K), rng.normal(size=K), 1e-5
        loss = lambda a: float((blk.layernorm(h + a * d, 0 * h, w + a * e, b + a * f, EPS)[0] * dy).sum())  # noqa: E731
        slope = (loss(t) - loss(-t)) / (2 * t)
        scale = np.abs(dx * d).sum() + np.abs(dw * e).sum() + np.abs(db * f).sum()
        assert abs(slope - (dx * d).sum() - (dw * e).sum() - (db * f).sum()) <= 2.0 ** -16 * scale


def test_layernorm_of_no_rows():
    e = torch.zeros(0, 256, dtype=BF, device="cuda")
    one, none = torch.ones(256, device="cuda"), torch.zeros(0, device="cuda")
    c, _ = dg().layernorm_fp8_1x128(e, one)
    dx, dw, db = dg().layernorm_backward(e, e, one, none, none, dweight=torch.full((256,), 9.0, device="cuda"),
                                         dbias=torch.full((256,), 9.0, device="cuda"))
    torch.cuda.synchronize()
    assert c.shape == dx.shape == (0, 256) and not dw.any() and not db.any()
