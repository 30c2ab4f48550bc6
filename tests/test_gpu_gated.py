"""GPU: the gated feed-forward product with FP8 output (dg_fp8_gemm_nt_gated_fp8) against the
oracle's exact product and the definitions in 64 bits (tests/_block64.py), and its backward
(dg_gated_backward_fp8). Integer-valued operands make gate and up exact in fp32, so that pre has
one possible value and h's distance is the activation's; N(0,1) operands add the product's own
error model. The shapes reach every kernel form: few rows and many, K splits, tail tiles, both
scale forms, odd M, one row, one K-block."""
import numpy as np
import pytest
import torch

import oracle
import synth
from tests import _block64 as blk
from tests import _ops64 as ops
from tests import gpu_util as gu
from tests.parity import MFMA_EPS, abs_product_sum
from tests.test_gpu_epilogue import operands, pack, product, small_values
from tests.test_gpu_norm import BF, F32, Fp8Out, hidden

pytestmark = pytest.mark.gpu

# M, I, K
SHAPES = [(1, 128, 128), (1, 2048, 512), (2, 384, 7168), (16, 4096, 1024), (17, 2048, 7168), (31, 640, 896),
          (33, 1152, 2048), (64, 2048, 7168), (64, 9216, 1024), (64, 256, 4224), (65, 128, 128), (100, 384, 384),
          (128, 1024, 2048), (130, 2048, 512), (200, 4096, 1664), (257, 1152, 1664), (500, 2048, 7168),
          (1000, 1024, 1024), (300, 2560, 4224), (2100, 2048, 2048), (700, 512, 5120)]


def dg():
    import fp8_block_scaled_dg_amd as m
    return m


def call(a, b, sa, sb, I, bias, act, packed_out, pre=None, what=""):
    M = a.shape[0]
    out = Fp8Out(M, I, packed_out)
    gu.announce(f"gated {what} M={M} I={I} K={a.shape[1]} act={act}")
    dg().fp8_gemm_nt_gated_fp8(a, b, sa, sb, bias=bias, activation=act, pre=pre, codes=out.codes, sf=out.sf)
    return out.result()


@pytest.mark.parametrize("M,I,K", SHAPES)
def test_gated_integers(M, I, K):
    A, B, sfA, sfB, r = operands(M, 2 * I, K, M + I + K)
    a, b, sa, sb = gu.codes(A), gu.codes(B), gu.dev(sfA), gu.dev(sfB)
    for act, bias_t, packed, keep in (("silu", BF, False, True), ("none", None, True, False), ("gelu", F32, True, True)):
        bias = small_values(1, 2 * I, bias_t) if bias_t else None
        pre = gu.Guarded((M, 2 * I), 6) if keep else None
        z = r + (bias.double().numpy() if bias_t else 0)
        assert np.array_equal(z.astype(np.float32), z), "the case is meant to be exact in fp32"
        first = None
        for _ in range(2):  # the counters of split K are back at zero
            codes, sf = call(a, b, pack(sfA) if packed else sa, sb, I, bias.cuda() if bias_t else None, act, packed,
                             pre.out if keep else None, f"bias={bias_t}")
            if keep:
                assert pre.guards_intact() and np.array_equal(pre.result(), oracle.bf16_rne(z)), "pre"
            assert first is None or all(np.array_equal(x, y) for x, y in zip(first, (codes, sf)))
            first = codes, sf
        h, dh = blk.gated(z, 0.0, act)
        blk.check_fp8(h, dh, codes, sf, f"{act} {M}x{I}x{K}")


@pytest.mark.parametrize("config", ["gated_m16", "gated_m32", "gated_m64", "pipe128x256"])
@pytest.mark.parametrize("M,I,K", [(1, 256, 128), (20, 384, 640), (64, 2048, 7168), (130, 512, 896), (33, 128, 7296),
                                   (300, 1152, 1920), (64, 7168, 7040)])
def test_gated_configurations(M, I, K, config, monkeypatch):
    # every kernel form, also where it would not be chosen: odd and even K-blocks, with and without
    # K splits, rows in several tiles, B streamed past the caches
    monkeypatch.setenv("DG_FORCE_CONFIG", config)
    assert config in dg().config_names()
    test_gated_integers(M, I, K)


@pytest.mark.parametrize("act", ["relu", "gelu_tanh"])
@pytest.mark.parametrize("M,I,K", [(5, 256, 896), (64, 2048, 2048), (257, 384, 640)])
def test_gated_other_activations(M, I, K, act):
    A, B, sfA, sfB, r = operands(M, 2 * I, K, M + I + K)
    codes, sf = call(gu.codes(A), gu.codes(B), gu.dev(sfA), gu.dev(sfB), I, None, act, False)
    h, dh = blk.gated(r, 0.0, act)
    blk.check_fp8(h, dh, codes, sf, f"{act} {M}x{I}x{K}")


@pytest.mark.parametrize("M,I,K", [(1, 1024, 2048), (48, 1152, 4096), (64, 512, 7168), (300, 1024, 3584), (1000, 2048, 1024)])
def test_gated_gaussian(M, I, K):
    rng = np.random.default_rng(M + I)
    N = 2 * I
    A, sfA = oracle.quantize_blocks(rng.normal(size=(M, K)).astype(np.float32), 1, 128)
    B, sfB = oracle.quantize_blocks((rng.normal(size=(N, K)) / np.sqrt(K)).astype(np.float32), 128, 128)
    r = product(A, B, sfA, sfB)
    dz = MFMA_EPS * abs_product_sum(A, B, sfA, sfB) + 2 * ops.U * np.abs(r)
    codes, sf = call(gu.codes(A), gu.codes(B), gu.dev(sfA), gu.dev(sfB), I, None, "silu", False)
    h, dh = blk.gated(r, dz, "silu")
    blk.check_fp8(h, dh, codes, sf, f"gaussian {M}x{I}x{K}")


def test_gated_is_the_unfused_product():
    # gate and up by the library's own GEMM with bf16 outputs give pre, bit for bit
    M, I, K = 200, 640, 1152
    A, B, sfA, sfB, r = operands(M, 2 * I, K, 3)
    a, b, sa, sb = gu.codes(A), gu.codes(B), gu.dev(sfA), gu.dev(sfB)
    c, pre = torch.empty(M, 2 * I, dtype=BF, device="cuda"), torch.empty(M, 2 * I, dtype=BF, device="cuda")
    dg().fp8_gemm_nt(a, b, c, sa, sb)
    c0, s0 = dg().fp8_gemm_nt_gated_fp8(a, b, sa, sb, pre=pre)
    c1, s1 = dg().fp8_gemm_nt_gated_fp8(a, b, sa, sb, ue8m0=True)
    torch.cuda.synchronize()
    assert torch.equal(c, pre) and torch.equal(c0.view(torch.uint8), c1.view(torch.uint8))
    assert s1.dtype == torch.int32 and s1.shape == (M, 2)


@pytest.mark.parametrize("M,I,K", [(1, 512, 1024), (40, 512, 1024), (200, 512, 1024)])
def test_gated_nothing_behind_the_rows_is_read(M, I, K):
    # A, B and the scales end with their buffers' last valid byte before NaN codes
    A, B, sfA, sfB, r = operands(M, 2 * I, K, 9)
    want = call(gu.codes(A), gu.codes(B), gu.dev(sfA), gu.dev(sfB), I, None, "silu", False)
    a2 = gu.codes(np.concatenate([A, np.full((64, K), 0x7F, np.uint8)]))[:M]
    b2 = gu.codes(np.concatenate([B, np.full((256, K), 0x7F, np.uint8)]))[:2 * I]
    sa2 = gu.dev(np.concatenate([sfA, np.full((64, K // 128), np.nan, np.float32)]))[:M]
    sb2 = gu.dev(np.concatenate([sfB, np.full((4, K // 128), np.nan, np.float32)]))[:2 * I // 128]
    got = call(a2, b2, sa2, sb2, I, None, "silu", False)
    assert all(np.array_equal(x, y) for x, y in zip(want, got))


def test_gated_empty_and_refused():
    z = lambda *s: torch.zeros(*s, dtype=torch.uint8, device="cuda")  # noqa: E731
    f = lambda *s: torch.ones(*s, device="cuda")  # noqa: E731
    c, s = dg().fp8_gemm_nt_gated_fp8(z(0, 256), z(256, 256), f(0, 2), f(2, 2))
    assert c.shape == (0, 128) and s.shape == (0, 1)
    with pytest.raises(ValueError, match="gate rows"):
        dg().fp8_gemm_nt_gated_fp8(z(4, 256), z(255, 256), f(4, 2), f(2, 2))
    with pytest.raises(dg().DGError, match="multiple of 128"):
        dg().fp8_gemm_nt_gated_fp8(z(4, 256), z(128, 256), f(4, 2), f(1, 2))
    with pytest.raises(ValueError, match="activation"):
        dg().fp8_gemm_nt_gated_fp8(z(4, 256), z(256, 256), f(4, 2), f(2, 2), activation="tanh")
    with pytest.raises(ValueError, match="bias has shape"):
        dg().fp8_gemm_nt_gated_fp8(z(4, 256), z(256, 256), f(4, 2), f(2, 2), bias=f(128))


# ---------------------------------------------------------------- backward

@pytest.mark.parametrize("M,I", [(1, 128), (1, 18432), (3, 384), (5, 1024), (130, 2048), (257, 1152), (4100, 256),
                                 (64, 7168), (130, 12288)])
@pytest.mark.parametrize("act", ops.ACTS)
def test_gated_backward(M, I, act):
    g = torch.Generator().manual_seed(M + I)
    dh = hidden(M * I, M, I, BF)
    pre = (2.5 * torch.randn(M, 2 * I, generator=g)).to(BF)
    pre.view(-1)[::97] = 0.0
    packed = act in ("silu", "none")
    out = Fp8Out(M, 2 * I, packed)
    db = torch.full((2 * I + 8,), 5.0, device="cuda")
    gu.announce(f"gated backward {act} M={M} I={I}")
    dg().gated_backward_fp8(dh.cuda(), pre.cuda(), act, codes=out.codes, sf=out.sf, dbias=db[4:2 * I + 4])
    codes, sf = out.result()
    assert torch.all(db[:4] == 5) and torch.all(db[-4:] == 5)
    p, dp = blk.gated_backward(dh.double().numpy(), pre.double().numpy(), act)
    blk.check_fp8(p, dp, codes, sf, f"{act} {M}x{I}")
    err = np.abs(db[4:2 * I + 4].double().cpu().numpy() - p.sum(0))
    assert np.all(err <= blk.COL * np.abs(p).sum(0) + dp.sum(0) + 1e-45), f"{act} dbias"


def test_gated_backward_forms_agree_and_empty():
    dh, pre = hidden(41, 300, 1152, BF).cuda(), hidden(42, 300, 2304, BF).cuda()
    c0, s0, db = dg().gated_backward_fp8(dh, pre, "gelu")
    c1, s1, none = dg().gated_backward_fp8(dh, pre, "gelu", need_dbias=False, ue8m0=True)
    c2, s2, db2 = dg().gated_backward_fp8(dh, pre, "gelu")
    e = torch.zeros(0, 256, dtype=BF, device="cuda")
    c3, _, db3 = dg().gated_backward_fp8(e, torch.zeros(0, 512, dtype=BF, device="cuda"),
                                         dbias=torch.full((512,), 9.0, device="cuda"))
    torch.cuda.synchronize()
    assert none is None and torch.equal(c0.view(torch.uint8), c1.view(torch.uint8))
    assert torch.equal(c0.view(torch.uint8), c2.view(torch.uint8)) and torch.equal(db, db2) and torch.equal(s0, s2)
    assert c3.shape == (0, 512) and not db3.any()


@pytest.mark.parametrize("act", ops.ACTS)
def test_gated_backward_values_of_every_size(act):
    # every finite bf16 gate: value and slope stay finite, and accurate where they do not underflow
    bits = np.arange(1 << 16, dtype=np.uint16)
    gate = torch.from_numpy(bits.view(np.int16)).view(BF)
    gate = gate[torch.isfinite(gate.float())]
    gate = torch.cat([gate, torch.zeros(-len(gate) % 128, dtype=BF)]).view(-1, 128)
    M = gate.shape[0]
    pre = torch.cat([gate, torch.ones(M, 128, dtype=BF)], 1).contiguous()
    gu.announce(f"gated backward, every gate, {act}")
    codes, sf, db = dg().gated_backward_fp8(torch.ones(M, 128, dtype=BF, device="cuda"), pre.cuda(), act)
    torch.cuda.synchronize()
    c, s = codes.view(torch.uint8).cpu().numpy(), sf.cpu().numpy()
    p, dp = blk.gated_backward(np.ones((M, 128)), pre.double().numpy(), act)
    blk.check_fp8(p, dp, c, s, act)
    assert torch.isfinite(db[:128]).all()


def test_gated_backward_past_32_bit_offsets():
    I = 8192
    M = (1 << 31) // I + 3  # 2^32 values of pre and more
    dh = torch.ones(M, I, dtype=BF, device="cuda")
    pre = torch.ones(M, 2 * I, dtype=BF, device="cuda")
    pre[-3:] = hidden(5, 3, 2 * I, BF).cuda()
    gu.announce(f"gated backward M={M} I={I}")
    codes, sf, _ = dg().gated_backward_fp8(dh, pre, "silu", need_dbias=False)
    c0, s0, _ = dg().gated_backward_fp8(dh[-3:].contiguous(), pre[-3:].contiguous(), "silu", need_dbias=False)
    torch.cuda.synchronize()
    assert torch.equal(codes[-3:].view(torch.uint8), c0.view(torch.uint8)) and torch.equal(sf[-3:], s0)
