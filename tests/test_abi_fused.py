"""CPU checks of the norm and epilogue calls' argument checks: refusals come from the host
before any HIP call, so fake addresses do, and the binding's own checks raise."""
import pytest

FAKE = 0x10000


@pytest.fixture(scope="module")
def dg():
    import fp8_block_scaled_dg_amd as m
    return m


def status(dg, code):
    return dg.lib.dg_status_string(code).decode()


def norm(dg, x=FAKE, r=FAKE, xt=1, w=FAKE, wt=1, eps=1e-6, h=FAKE, rstd=FAKE, codes=FAKE, sf=FAKE,
         packed=0, M=4, K=256):
    return status(dg, dg.lib.dg_rmsnorm_fp8_1x128(x, r, xt, w, wt, eps, h, rstd, codes, sf, packed,
                                                  M, K, None))


def norm_bwd(dg, dy=FAKE, dh=FAKE, h=FAKE, xt=1, w=FAKE, wt=1, rstd=FAKE, dx=FAKE, dw=FAKE, M=4, K=256):
    return status(dg, dg.lib.dg_rmsnorm_backward(dy, dh, h, xt, w, wt, rstd, dx, dw, M, K, None))


def gemm(dg, A=FAKE, B=FAKE, C=FAKE, sA=FAKE, packed=0, sB=FAKE, bias=FAKE, bt=1, act=2, res=FAKE,
         pre=FAKE, M=64, N=128, K=256):
    return status(dg, dg.lib.dg_fp8_gemm_nt_bias_act(A, B, C, sA, packed, sB, bias, bt, act, res, pre,
                                                     M, N, K, None))


def gemm_fp8(dg, A=FAKE, B=FAKE, codes=FAKE, sf=FAKE, sp=0, sA=FAKE, packed=0, sB=FAKE, bias=FAKE,
             bt=1, act=2, pre=FAKE, M=64, N=128, K=256):
    return status(dg, dg.lib.dg_fp8_gemm_nt_bias_act_fp8(A, B, codes, sf, sp, sA, packed, sB, bias, bt,
                                                         act, pre, M, N, K, None))


def act_bwd(dg, dc=FAKE, pre=FAKE, act=2, codes=FAKE, sf=FAKE, packed=0, dbias=FAKE, M=4, N=256):
    return status(dg, dg.lib.dg_bias_act_backward_fp8(dc, pre, act, codes, sf, packed, dbias, M, N, None))


@pytest.mark.parametrize("call", [norm, norm_bwd])
def test_norm_calls_refuse(dg, call):
    assert call(dg, K=200) == "DG_ERR_BAD_SHAPE"
    assert call(dg, M=-1) == "DG_ERR_BAD_SHAPE"
    assert call(dg, K=-128) == "DG_ERR_BAD_SHAPE"
    assert call(dg, xt=2) == "DG_ERR_BAD_SHAPE"
    assert call(dg, wt=-1) == "DG_ERR_BAD_SHAPE"
    assert call(dg, w=None) == "DG_ERR_NULL_POINTER"
    assert call(dg, w=FAKE + 8) == "DG_ERR_MISALIGNED"
    assert call(dg, h=FAKE + 8) == "DG_ERR_MISALIGNED"
    assert call(dg, rstd=FAKE + 2) == "DG_ERR_MISALIGNED"
    assert call(dg, K=32768 + 128) == "DG_ERR_UNSUPPORTED_SHAPE"
    assert call(dg, M=1 << 33, K=1 << 10) == "DG_ERR_UNSUPPORTED_SHAPE"
    assert call(dg, K=0) == "DG_OK"


def test_norm_refuses(dg):
    for eps in (0.0, -1e-6, float("inf"), float("nan")):
        assert norm(dg, eps=eps) == "DG_ERR_BAD_SHAPE"
    for name in ("x", "codes", "sf"):
        assert norm(dg, **{name: None}) == "DG_ERR_NULL_POINTER"
    for name in ("x", "r", "codes"):
        assert norm(dg, **{name: FAKE + 8}) == "DG_ERR_MISALIGNED"
    assert norm(dg, sf=FAKE + 2) == "DG_ERR_MISALIGNED"
    assert norm(dg, x=None, w=None, codes=None, sf=None, M=0) == "DG_OK"


def test_norm_backward_refuses(dg):
    for name in ("dy", "h", "rstd", "dx", "dw"):
        assert norm_bwd(dg, **{name: None}) == "DG_ERR_NULL_POINTER"
    for name in ("dy", "dh", "dx", "dw"):
        assert norm_bwd(dg, **{name: FAKE + 8}) == "DG_ERR_MISALIGNED"
    assert norm_bwd(dg, dw=None, M=0) == "DG_ERR_NULL_POINTER"


@pytest.mark.parametrize("call", [gemm, gemm_fp8])
def test_gemm_calls_refuse(dg, call):
    for name in ("A", "B", "sA", "sB"):
        assert call(dg, **{name: None}) == "DG_ERR_NULL_POINTER"
    for name in ("A", "B", "bias", "pre"):
        assert call(dg, **{name: FAKE + 8}) == "DG_ERR_MISALIGNED"
    for bad in (dict(K=200), dict(K=0), dict(M=-1), dict(N=120), dict(N=-128), dict(act=5), dict(act=-1),
                dict(bt=2)):
        assert call(dg, **bad) == "DG_ERR_BAD_SHAPE", bad
    assert call(dg, M=65, K=(1 << 22) + 128) == "DG_ERR_UNSUPPORTED_SHAPE"
    assert call(dg, M=(1 << 30) + 1) == "DG_ERR_UNSUPPORTED_SHAPE"
    assert call(dg, M=0, A=None, B=None, sA=None, sB=None) == "DG_OK"
    assert call(dg, N=0, A=None, B=None, sA=None, sB=None) == "DG_OK"


def test_gemm_output_refusals(dg):
    assert gemm(dg, C=None) == "DG_ERR_NULL_POINTER"
    assert gemm(dg, res=FAKE + 8) == "DG_ERR_MISALIGNED"
    assert gemm_fp8(dg, codes=None) == "DG_ERR_NULL_POINTER"
    assert gemm_fp8(dg, sf=None) == "DG_ERR_NULL_POINTER"
    assert gemm_fp8(dg, codes=FAKE + 8) == "DG_ERR_MISALIGNED"
    assert gemm_fp8(dg, sf=FAKE + 2) == "DG_ERR_MISALIGNED"
    assert gemm_fp8(dg, N=2112) == "DG_ERR_BAD_SHAPE"  # not a whole number of 1x128 blocks


def test_act_backward_refuses(dg):
    for name in ("dc", "pre", "codes", "sf"):
        assert act_bwd(dg, **{name: None}) == "DG_ERR_NULL_POINTER"
    for name in ("dc", "pre", "codes", "dbias"):
        assert act_bwd(dg, **{name: FAKE + 8}) == "DG_ERR_MISALIGNED"
    assert act_bwd(dg, sf=FAKE + 2) == "DG_ERR_MISALIGNED"
    assert act_bwd(dg, N=200) == "DG_ERR_BAD_SHAPE"
    assert act_bwd(dg, M=-1) == "DG_ERR_BAD_SHAPE"
    assert act_bwd(dg, act=9) == "DG_ERR_BAD_SHAPE"
    assert act_bwd(dg, M=1 << 33, N=1 << 10) == "DG_ERR_UNSUPPORTED_SHAPE"
    assert act_bwd(dg, M=0, dc=None, pre=None, codes=None, sf=None, dbias=None) == "DG_OK"
    assert act_bwd(dg, N=0) == "DG_OK"


def test_binding_refuses(dg):
    import torch
    bf, f8 = torch.bfloat16, torch.float8_e4m3fn
    x = torch.zeros(2, 128, dtype=bf)
    w = torch.ones(128)
    with pytest.raises(TypeError):
        dg.rmsnorm_fp8_1x128(x.half(), w)
    with pytest.raises(ValueError):
        dg.rmsnorm_fp8_1x128(x, w)  # not on a GPU
    with pytest.raises(ValueError):
        dg.rmsnorm_fp8_1x128(x[0], w)
    with pytest.raises(ValueError):
        dg.rmsnorm_backward(x, x, w, torch.ones(2))
    a, b = torch.zeros(2, 128, dtype=f8), torch.zeros(128, 128, dtype=f8)
    with pytest.raises(TypeError):
        dg.fp8_gemm_nt_bias_act(a.float(), b, x, torch.ones(2, 1), torch.ones(1, 1))
    with pytest.raises(ValueError):
        dg.fp8_gemm_nt_bias_act_fp8(a, b, torch.ones(2, 1), torch.ones(1, 1))
    with pytest.raises(ValueError):
        dg._act("swish")
    with pytest.raises(ValueError):
        dg.bias_act_backward_fp8(x, x, "relu")


@pytest.mark.gpu
def test_binding_refuses_shapes_and_strides(dg):
    import torch
    bf, f8, d = torch.bfloat16, torch.float8_e4m3fn, "cuda"
    x, w = torch.zeros(4, 256, dtype=bf, device=d), torch.ones(256, device=d)
    with pytest.raises(ValueError):
        dg.rmsnorm_fp8_1x128(x[:, :128], w[:128])                      # rows apart
    with pytest.raises(ValueError):
        dg.rmsnorm_fp8_1x128(x, w[:128])
    with pytest.raises(TypeError):
        dg.rmsnorm_fp8_1x128(x, w, residual=x.float())
    with pytest.raises(TypeError):
        dg.rmsnorm_fp8_1x128(x, w, h=torch.zeros(4, 256, device=d))
    with pytest.raises(ValueError):
        dg.rmsnorm_fp8_1x128(x, w, sf=torch.zeros(4, 2, dtype=torch.int32, device=d))
    with pytest.raises(dg.DGError):
        dg.rmsnorm_fp8_1x128(x, w, eps=0.0)
    with pytest.raises(dg.DGError):
        dg.rmsnorm_fp8_1x128(torch.zeros(4, 200, dtype=bf, device=d), torch.ones(200, device=d))
    with pytest.raises(TypeError):
        dg.rmsnorm_backward(x.float(), x, w, torch.ones(4, device=d))
    a, b = torch.zeros(4, 128, dtype=f8, device=d), torch.zeros(256, 128, dtype=f8, device=d)
    sa, sb = torch.ones(4, 1, device=d), torch.ones(2, 1, device=d)
    with pytest.raises(ValueError):
        dg.fp8_gemm_nt_bias_act(a, b, x, sa, sb, bias=w[:128])
    with pytest.raises(TypeError):
        dg.fp8_gemm_nt_bias_act(a, b, x, sa, sb, bias=w.half())
    with pytest.raises(TypeError):
        dg.fp8_gemm_nt_bias_act(a, b, x, sa, sb, residual=x.float())
    with pytest.raises(ValueError):
        dg.fp8_gemm_nt_bias_act(a, b, x, sa, sb, pre=x[:2])
    with pytest.raises(ValueError):
        dg.fp8_gemm_nt_bias_act(a, b, x, sa, sb, activation="tanh")
    with pytest.raises(dg.DGError):
        dg.bias_act_backward_fp8(x, None, "relu")                       # needs pre
    with pytest.raises(dg.DGError):                                      # misaligned view
        dg.bias_act_backward_fp8(torch.zeros(257, dtype=bf, device=d)[1:].view(1, 256), need_dbias=False)
