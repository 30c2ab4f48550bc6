"""GPU: the dense GEMM with bias, activation and residual in its epilogue
(dg_fp8_gemm_nt_bias_act) and with an FP8 output (dg_fp8_gemm_nt_bias_act_fp8), against the
oracle's exact product and the definitions in 64 bits (tests/_ops64.py).

Integer-valued operands make the product exact in fp32, so that without an activation the
bf16 output has one possible value (bias and residual chosen so that their sums are exact
too), and with one its distance is the activation's. N(0,1) operands add the product's own
error model. Every kernel that serves the calls is reached: the M <= 64 kernel in each of
its forms, with and without split K, the compute-bound kernel's tiles, its K-split tail
tiles, both scale forms; odd M, N tails inside a tile, one row, one K-block."""
import numpy as np
import pytest
import torch

import oracle
import synth
from tests import _ops64 as ops
from tests import gpu_util as gu
from tests.parity import MFMA_EPS, abs_product_sum, bf16_to_f64
from tests.test_gpu_norm import Fp8Out
from tests.test_gpu_parity import int_operands
from tests.test_gpu_swiglu import check

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32

SHAPES = [(1, 256, 128), (1, 2048, 512), (17, 2112, 7168), (64, 4096, 7168), (33, 1040, 2048),
          (64, 256, 896), (5, 32768, 512), (64, 18432, 1024), (65, 128, 128), (100, 272, 384),
          (128, 1040, 2048), (130, 4096, 512), (257, 2112, 1664), (1000, 4096, 1024), (300, 5120, 4224),
          (2100, 4096, 2048)]
FP8_SHAPES = [s if s[1] % 128 == 0 else (s[0], s[1] // 128 * 128, s[2]) for s in SHAPES]


def dg():
    import fp8_block_scaled_dg_amd as m
    return m


def product(A, B, sfA, sfB):
    """The block-scaled product of integer-valued operands: exact in fp64 in any order."""
    vals = torch.from_numpy(np.nan_to_num(oracle.e4m3fn_values())).cuda()
    a = vals[torch.from_numpy(A).cuda().long()] * gu.dev(sfA).double().repeat_interleave(128, 1)
    b = vals[torch.from_numpy(B).cuda().long()]
    b = b * gu.dev(sfB).double().repeat_interleave(128, 1).repeat_interleave(128, 0)[:B.shape[0]]
    return (a @ b.t().contiguous()).cpu().numpy()


def operands(M, N, K, seed, size=2.0):
    """Integer-valued codes with power-of-two scales, and the product, of size about `size`."""
    rng = np.random.default_rng(seed)
    A, B, sfA, sfB = int_operands(rng, M, N, K)
    r = product(A, B, sfA, sfB)
    e = int(np.round(np.log2(size / max(1e-30, np.std(r)))))
    return A, B, sfA, np.ldexp(sfB, e).astype(np.float32), np.ldexp(r, e)


def pack(sfA):
    """fp32 power-of-two scales to packed words."""
    M, KB = sfA.shape
    b = np.zeros((M, (KB + 3) // 4 * 4), np.uint8)
    b[:, :KB] = np.frexp(sfA)[1] - 1 + 127
    return torch.from_numpy(b.view(np.int32)).cuda()


def small_values(seed, shape, dtype, step=2.0 ** -4):
    """Multiples of step up to 8: sums with the products stay exact in fp32."""
    rng = np.random.default_rng(seed)
    return torch.from_numpy(rng.integers(-127, 128, size=shape) * step).to(dtype)


@pytest.mark.parametrize("M,N,K", SHAPES)
def test_bias_and_residual_bitwise(M, N, K):
    A, B, sfA, sfB, r = operands(M, N, K, M + N + K)
    a, b, sa, sb = gu.codes(A), gu.codes(B), gu.dev(sfA), gu.dev(sfB)
    for bias_t, res, packed in ((BF, True, False), (F32, False, True), (None, True, True)):
        bias = small_values(1, N, bias_t) if bias_t else None
        residual = small_values(2, (M, N), BF) if res else None
        out = gu.Guarded((M, N), 5)
        pre = gu.Guarded((M, N), 6)
        gu.announce(f"bias_act M={M} N={N} K={K} bias={bias_t} residual={res} packed={packed}")
        dg().fp8_gemm_nt_bias_act(a, b, out.out, pack(sfA) if packed else sa, sb,
                                  bias=bias.cuda() if bias_t else None,
                                  residual=residual.cuda() if res else None, pre=pre.out)
        torch.cuda.synchronize()
        assert out.guards_intact() and pre.guards_intact(), "write outside an output"
        z = r + (bias.double().numpy() if bias_t else 0)
        c = z + (residual.double().numpy() if res else 0)
        assert np.array_equal(c.astype(np.float32), c), "the case is meant to be exact in fp32"
        assert np.array_equal(pre.result(), oracle.bf16_rne(z)), "pre"
        assert np.array_equal(out.result(), oracle.bf16_rne(c)), "c"


@pytest.mark.parametrize("M,N,K", [(1, 16512, 6272), (16, 20464, 5120), (17, 18432, 5760), (33, 24576, 4224),
                                   (64, 16640, 6400), (64, 32640, 3200)])
def test_large_b_bitwise(M, N, K):
    # 129 to 255 column tiles of a B of about 100 MB, with up to 64 rows
    A, B, sfA, sfB, r = operands(M, N, K, M + N + K)
    bias, residual = small_values(1, N, BF), small_values(2, (M, N), BF)
    out, pre = gu.Guarded((M, N), 5), gu.Guarded((M, N), 6)
    args = (gu.codes(A), gu.codes(B), out.out, gu.dev(sfA), gu.dev(sfB))
    gu.announce(f"large B M={M} N={N} K={K}")
    for _ in range(2):
        out.out.zero_(), pre.out.zero_()
        dg().fp8_gemm_nt_bias_act(*args, bias=bias.cuda(), residual=residual.cuda(), pre=pre.out)
        torch.cuda.synchronize()
        assert out.guards_intact() and pre.guards_intact(), "write outside an output"
        z = r + bias.double().numpy()
        c = z + residual.double().numpy()
        assert np.array_equal(c.astype(np.float32), c), "the case is meant to be exact in fp32"
        assert np.array_equal(pre.result(), oracle.bf16_rne(z)), "pre"
        assert np.array_equal(out.result(), oracle.bf16_rne(c)), "c"


@pytest.mark.parametrize("M,N,K", [(17, 2112, 7168), (64, 256, 896), (130, 4096, 512), (1000, 1040, 1024)])
@pytest.mark.parametrize("act", ops.ACTS[1:])
def test_activation(M, N, K, act):
    A, B, sfA, sfB, r = operands(M, N, K, M + N + K)
    bias, residual = small_values(3, N, BF), small_values(4, (M, N), BF)
    out = gu.Guarded((M, N), 7)
    gu.announce(f"bias_act {act} M={M} N={N} K={K}")
    dg().fp8_gemm_nt_bias_act(gu.codes(A), gu.codes(B), out.out, gu.dev(sfA), gu.dev(sfB), bias=bias.cuda(),
                              activation=act, residual=residual.cuda())
    torch.cuda.synchronize()
    assert out.guards_intact()
    z = r + bias.double().numpy()
    c = ops.act(z, act) + residual.double().numpy()
    d = ops.act_bound(z, 0.0, act) + 2 * ops.U * np.abs(c)
    err = np.abs(bf16_to_f64(out.result()) - c)
    assert np.all(err <= d + ops.bf16_slack(np.abs(c) + d)), f"{act}: {np.max(err / (d + ops.bf16_slack(c)))}"


@pytest.mark.parametrize("act", ops.ACTS)
def test_gelu_tails_and_slopes_of_every_size(act):
    """A product that is one code times one code: the activation over its whole range."""
    vals = oracle.e4m3fn_values()
    codes = np.array([c for c in range(256) if np.isfinite(vals[c])], dtype=np.uint8)
    N, K = 256, 128
    A, B = np.zeros((16, K), np.uint8), np.zeros((N, K), np.uint8)
    A[:, 0] = 0x38  # 1.0
    B[:codes.size, 0] = codes
    sfA = np.ldexp(1.0, np.arange(-14, 2)).astype(np.float32)[:, None]
    sfB = np.ones((2, 1), np.float32)
    z = vals[A[:, :1]].astype(np.float64) * sfA * np.nan_to_num(vals[B[:, 0]])[None, :]
    c = torch.empty(16, N, dtype=BF, device="cuda")
    dg().fp8_gemm_nt_bias_act(gu.codes(A), gu.codes(B), c, gu.dev(sfA), gu.dev(sfB), activation=act)
    want = ops.act(z, act)
    d = ops.act_bound(z, 0.0, act)
    err = np.abs(c.double().cpu().numpy() - want)
    assert np.all(err <= d + ops.bf16_slack(np.abs(want) + d)), act


@pytest.mark.parametrize("M,N,K", FP8_SHAPES)
def test_fp8_output(M, N, K):
    A, B, sfA, sfB, r = operands(M, N, K, M + N + K)
    a, b, sa, sb = gu.codes(A), gu.codes(B), gu.dev(sfA), gu.dev(sfB)
    bias = small_values(8, N, BF)
    z = r + bias.double().numpy()
    for act, sp, packed, keep in (("none", False, True, True), ("gelu", True, False, False)):
        out = Fp8Out(M, N, sp)
        pre = gu.Guarded((M, N), 9)
        gu.announce(f"bias_act_fp8 {act} M={M} N={N} K={K}")
        dg().fp8_gemm_nt_bias_act_fp8(a, b, pack(sfA) if packed else sa, sb, bias=bias.cuda(), activation=act,
                                      pre=pre.out if keep else None, codes=out.codes, sf=out.sf)
        codes, sf = out.result()
        assert pre.guards_intact()
        if keep:
            assert np.array_equal(pre.result(), oracle.bf16_rne(z)), "pre"
        if act == "none":  # exact in fp32: the oracle quantizer's bytes
            rc, rs = oracle.quantize_blocks(z.astype(np.float32), 1, 128)
            assert np.array_equal(rs, sf) and np.array_equal(rc, codes)
        else:
            h = ops.act(z, act)
            check(h, ops.act_bound(z, 0.0, act), codes, sf, f"{act} {M}x{N}x{K}", strict=False)


@pytest.mark.parametrize("M,N,K", [(64, 2048, 7168), (64, 32768, 512), (300, 2048, 4096)])
def test_normal_operands(M, N, K):
    """N(0,1) operands: the product's error model carried through gelu."""
    A, sfA = oracle.quantize_blocks(synth.normal_rows(1, M, K), 1, 128)
    B, sfB = oracle.quantize_blocks(synth.normal_rows(2, N, K) / np.sqrt(K), 128, 128)
    r, ra = oracle.gemm_nt(A, B, sfA, sfB), abs_product_sum(A, B, sfA, sfB)
    bias, residual = small_values(10, N, F32), small_values(11, (M, N), BF)
    z = r + bias.double().numpy()
    c = ops.act(z, "gelu") + residual.double().numpy()
    d = ops.act_bound(z, MFMA_EPS * ra + 2 * ops.U * np.abs(z), "gelu") + 2 * ops.U * np.abs(c)
    out = gu.Guarded((M, N), 12)
    a, b, sa, sb = gu.codes(A), gu.codes(B), gu.dev(sfA), gu.dev(sfB)
    dg().fp8_gemm_nt_bias_act(a, b, out.out, sa, sb, bias=bias.cuda(), activation="gelu",
                              residual=residual.cuda())
    torch.cuda.synchronize()
    err = np.abs(bf16_to_f64(out.result()) - c)
    assert out.guards_intact() and np.all(err <= d + ops.bf16_slack(np.abs(c) + d))
    fp8 = Fp8Out(M, N, True)
    dg().fp8_gemm_nt_bias_act_fp8(a, b, sa, sb, bias=bias.cuda(), activation="gelu", codes=fp8.codes, sf=fp8.sf)
    codes, sf = fp8.result()
    check(ops.act(z, "gelu"), ops.act_bound(z, MFMA_EPS * ra + 2 * ops.U * np.abs(z), "gelu"), codes, sf,
          f"normal {M}x{N}x{K}", strict=False)


@pytest.mark.parametrize("config", ["ring_n64", "ring_n128", "ring_n128_wide"])
@pytest.mark.parametrize("M", [1, 15, 16, 17, 32, 33, 64])
@pytest.mark.parametrize("N,KB", [(128, 1), (256, 2), (384, 3), (128, 5), (1040, 6), (512, 7), (256, 13), (128, 40)])
def test_row_counts_and_run_lengths(monkeypatch, config, M, N, KB):
    """The M <= 64 kernel: every number of 16-row tiles, runs of K-blocks that end in each
    stage of its ring, with and without an odd last block, and N tails."""
    monkeypatch.setenv("DG_FORCE_CONFIG", config)
    fp8 = config != "ring_n64" and N % 128 == 0
    packed = (M + KB) % 2 == 0
    A, B, sfA, sfB, r = operands(M, N, 128 * KB, M + N + KB)
    a, b, sa, sb = gu.codes(A), gu.codes(B), pack(sfA) if packed else gu.dev(sfA), gu.dev(sfB)
    out = gu.Guarded((M, N), 5)
    gu.announce(f"{config} M={M} N={N} KB={KB}")
    dg().fp8_gemm_nt_bias_act(a, b, out.out, sa, sb)
    torch.cuda.synchronize()
    assert out.guards_intact() and np.array_equal(out.result(), oracle.bf16_rne(r))
    if fp8:
        out = Fp8Out(M, N, not packed)
        gu.announce(f"{config} FP8 M={M} N={N} KB={KB}")
        dg().fp8_gemm_nt_bias_act_fp8(a, b, sa, sb, codes=out.codes, sf=out.sf)
        codes, sf = out.result()
        rc, rs = oracle.quantize_blocks(r.astype(np.float32), 1, 128)
        assert np.array_equal(rs, sf) and np.array_equal(rc, codes)


@pytest.mark.parametrize("config", ["ring_n64", "ring_n128", "ring_m128_n128", "pipe128x256", "pipe256x128"])
@pytest.mark.parametrize("M,N,KB", [(65, 128, 1), (127, 384, 4), (129, 256, 5), (200, 640, 12), (300, 1040, 7),
                                    (257, 128, 40), (700, 2176, 3)])
def test_row_tiles(monkeypatch, config, M, N, KB):
    """Several row tiles, a ragged last one, with and without split K, on each kernel that
    the choice by estimated time may take."""
    monkeypatch.setenv("DG_FORCE_CONFIG", config)
    packed = (M + KB) % 2 == 0
    A, B, sfA, sfB, r = operands(M, N, 128 * KB, M + N + KB)
    a, b, sa, sb = gu.codes(A), gu.codes(B), pack(sfA) if packed else gu.dev(sfA), gu.dev(sfB)
    residual = small_values(23, (M, N), BF)
    out, pre = gu.Guarded((M, N), 5), gu.Guarded((M, N), 6)
    gu.announce(f"{config} M={M} N={N} KB={KB}")
    dg().fp8_gemm_nt_bias_act(a, b, out.out, sa, sb, residual=residual.cuda(), pre=pre.out)
    torch.cuda.synchronize()
    assert out.guards_intact() and np.array_equal(out.result(), oracle.bf16_rne(r + residual.double().numpy()))
    assert pre.guards_intact() and np.array_equal(pre.result(), oracle.bf16_rne(r))
    if N % 128 == 0 and config != "ring_n64":
        fp8 = Fp8Out(M, N, not packed)
        gu.announce(f"{config} FP8 M={M} N={N} KB={KB}")
        dg().fp8_gemm_nt_bias_act_fp8(a, b, sa, sb, codes=fp8.codes, sf=fp8.sf)
        codes, sf = fp8.result()
        rc, rs = oracle.quantize_blocks(r.astype(np.float32), 1, 128)
        assert np.array_equal(rs, sf) and np.array_equal(rc, codes)


@pytest.mark.parametrize("M,N,K", [(130, 2112, 2048), (1000, 1024, 512)])
def test_plain_call_and_no_epilogue_agree(monkeypatch, M, N, K):
    monkeypatch.setenv("DG_FORCE_CONFIG", "pipe128x256")
    # nothing to add: the same bits as the plain call, whose kernel this is
    rng = np.random.default_rng(13)
    A, sfA = oracle.quantize_blocks(rng.normal(size=(M, K)).astype(np.float32), 1, 128)
    B, sfB = oracle.quantize_blocks(rng.normal(size=(N, K)).astype(np.float32), 128, 128)
    a, b, sa, sb = gu.codes(A), gu.codes(B), gu.dev(sfA), gu.dev(sfB)
    c0, c1 = (torch.empty(M, N, dtype=BF, device="cuda") for _ in range(2))
    dg().fp8_gemm_nt(a, b, c0, sa, sb)
    dg().fp8_gemm_nt_bias_act(a, b, c1, sa, sb)
    torch.cuda.synchronize()
    assert torch.equal(c0, c1)


@pytest.mark.parametrize("M,N,K", [(64, 2112, 7168), (7, 4096, 512), (300, 2112, 2048), (1000, 4096, 1024)])
def test_residual_in_place(M, N, K):
    A, B, sfA, sfB, r = operands(M, N, K, 14)
    residual = small_values(15, (M, N), BF)
    c = residual.cuda()
    dg().fp8_gemm_nt_bias_act(gu.codes(A), gu.codes(B), c, gu.dev(sfA), gu.dev(sfB), residual=c)
    torch.cuda.synchronize()
    assert np.array_equal(gu.bits(c), oracle.bf16_rne(r + residual.double().numpy()))


def test_nan_and_infinity_pass_through():
    A, B, sfA, sfB, r = operands(70, 512, 256, 16)
    bias = torch.zeros(512)
    bias[3], bias[400] = float("nan"), float("inf")
    residual = torch.zeros(70, 512, dtype=BF)
    residual[5, 10], residual[6, 400] = float("nan"), float("-inf")
    for act in ops.ACTS:
        c = torch.empty(70, 512, dtype=BF, device="cuda")
        dg().fp8_gemm_nt_bias_act(gu.codes(A), gu.codes(B), c, gu.dev(sfA), gu.dev(sfB), bias=bias.cuda(),
                                  activation=act, residual=residual.cuda())
        got = c.float().cpu()
        nan = torch.zeros(70, 512, dtype=torch.bool)
        nan[:, 3] = nan[5, 10] = nan[6, 400] = True
        assert torch.equal(torch.isnan(got), nan), act
        inf = torch.zeros(70, 512, dtype=torch.bool)
        inf[:, 400] = True
        inf[6, 400] = False
        assert torch.equal(torch.isinf(got), inf), act


def test_no_rows_and_no_columns():
    f8 = torch.float8_e4m3fn
    a, b = torch.zeros(0, 256, dtype=f8, device="cuda"), torch.zeros(128, 256, dtype=f8, device="cuda")
    sa, sb = torch.ones(0, 2, device="cuda"), torch.ones(1, 2, device="cuda")
    dg().fp8_gemm_nt_bias_act(a, b, torch.empty(0, 128, dtype=BF, device="cuda"), sa, sb)
    codes, sf = dg().fp8_gemm_nt_bias_act_fp8(a, b, sa, sb)
    torch.cuda.synchronize()
    assert codes.shape == (0, 128) and sf.shape == (0, 1)


def test_rows_past_32_bit_offsets():
    # C and codes of over 2^31 values: the last rows equal those of a small call
    M, N, K = 66000, 32768, 128
    g = torch.Generator(device="cuda").manual_seed(1)
    a = torch.randint(0, 0x70, (M, K), generator=g, device="cuda", dtype=torch.uint8).view(torch.float8_e4m3fn)
    b = torch.randint(0, 0x70, (N, K), generator=g, device="cuda", dtype=torch.uint8).view(torch.float8_e4m3fn)
    sa = torch.rand(M, 1, generator=g, device="cuda") + 0.5
    sb = torch.rand(N // 128, 1, generator=g, device="cuda") * 2.0 ** -8
    res = torch.randn(M, N, generator=g, device="cuda", dtype=BF)
    c = torch.empty(M, N, dtype=BF, device="cuda")
    gu.announce(f"bias_act M={M} N={N} K={K}")
    dg().fp8_gemm_nt_bias_act(a, b, c, sa, sb, activation="silu", residual=res)
    codes, sf = dg().fp8_gemm_nt_bias_act_fp8(a, b, sa, sb, activation="silu")
    t = slice(M - 200, M)
    c0 = torch.empty(200, N, dtype=BF, device="cuda")
    at, st = a[t].contiguous(), sa[t].contiguous()
    dg().fp8_gemm_nt_bias_act(at, b, c0, st, sb, activation="silu", residual=res[t].contiguous())
    codes0, sf0 = dg().fp8_gemm_nt_bias_act_fp8(at, b, st, sb, activation="silu")
    torch.cuda.synchronize()
    assert torch.equal(c[t], c0)
    assert torch.equal(codes[t].view(torch.uint8), codes0.view(torch.uint8)) and torch.equal(sf[t], sf0)


@pytest.mark.parametrize("M,N,K", [(64, 2048, 7168), (384, 768, 2048)])
def test_graph_replays_match_eager(M, N, K):
    A, B, sfA, sfB, _ = operands(M, N, K, 17)
    a, b, sa, sb = gu.codes(A), gu.codes(B), gu.dev(sfA), gu.dev(sfB)
    bias, residual = small_values(18, N, BF).cuda(), small_values(19, (M, N), BF).cuda()
    x, w = torch.randn(M, N, device="cuda").to(BF), torch.ones(N, device="cuda")
    c, pre, h = (torch.empty(M, N, dtype=BF, device="cuda") for _ in range(3))
    dx, dw, db, rstd = torch.empty_like(x), *(torch.empty(n, device="cuda") for n in (N, N, M))
    o1, o2, o3 = (Fp8Out(M, N, p, 30 + 2 * i) for i, p in enumerate((True, False, True)))
    outs = [c, pre, h, dx, dw, db, rstd] + [t for o in (o1, o2, o3) for t in (o.codes.view(torch.uint8), o.sf)]

    def step():
        dg().rmsnorm_fp8_1x128(x, w, residual=residual, h=h, rstd=rstd, codes=o1.codes, sf=o1.sf)
        dg().fp8_gemm_nt_bias_act(a, b, c, sa, sb, bias=bias, activation="gelu", residual=residual)
        dg().fp8_gemm_nt_bias_act_fp8(a, b, sa, sb, bias=bias, activation="silu", pre=pre, codes=o2.codes, sf=o2.sf)
        dg().bias_act_backward_fp8(c, pre, "silu", codes=o3.codes, sf=o3.sf, dbias=db)
        dg().rmsnorm_backward(c, h, w, rstd, dh=x, dx=dx, dweight=dw)

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
    torch.cuda.synchronize()
    want = [t.clone() for t in outs]
    g = torch.cuda.CUDAGraph()
    gu.announce(f"graph of the norm and epilogue calls {M}x{N}x{K}")
    with torch.cuda.graph(g, stream=s):
        step()
    for rep in range(4):
        for t in outs:
            t.zero_()
        torch.cuda.synchronize()
        with torch.cuda.stream(s):
            g.replay()
        torch.cuda.synchronize()
        for i, (t, v) in enumerate(zip(outs, want)):
            assert torch.equal(t, v), f"replay {rep}, output {i}"
        with torch.cuda.stream(s):  # eager calls of other shapes between the replays
            dg().rmsnorm_backward(x[:3].contiguous(), h[:3].contiguous(), w, rstd[:3].contiguous())
            dg().fp8_gemm_nt(a[:1].contiguous(), b, torch.empty(1, N, dtype=BF, device="cuda"),
                             sa[:1].contiguous(), sb)
        torch.cuda.synchronize()
