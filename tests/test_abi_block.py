"""CPU checks of the argument checks of the layer norm, the gated product and dropout:
refusals come from the host before any HIP call, so fake addresses do, and the binding's own
checks raise."""
import pytest
import torch

FAKE = 0x10000


@pytest.fixture(scope="module")
def dg():
    import fp8_block_scaled_dg_amd as m
    return m


def status(dg, code):
    return dg.lib.dg_status_string(code).decode()


def norm(dg, x=FAKE, r=FAKE, xt=1, w=FAKE, b=FAKE, wt=1, eps=1e-5, p=0.1, rng=FAKE, sub=0, h=FAKE, mean=FAKE,
         rstd=FAKE, codes=FAKE, sf=FAKE, packed=0, M=4, K=256):
    return status(dg, dg.lib.dg_layernorm_fp8_1x128(x, r, xt, w, b, wt, eps, p, rng, sub, h, mean, rstd, codes,
                                                    sf, packed, M, K, None))


def norm_bwd(dg, dy=FAKE, dh=FAKE, h=FAKE, xt=1, w=FAKE, wt=1, mean=FAKE, rstd=FAKE, dx=FAKE, dw=FAKE, db=FAKE,
             M=4, K=256):
    return status(dg, dg.lib.dg_layernorm_backward(dy, dh, h, xt, w, wt, mean, rstd, dx, dw, db, M, K, None))


def gated(dg, A=FAKE, B=FAKE, codes=FAKE, sf=FAKE, sp=0, sA=FAKE, packed=0, sB=FAKE, bias=FAKE, bt=1, act=2,
          pre=FAKE, M=64, I=128, K=256):
    return status(dg, dg.lib.dg_fp8_gemm_nt_gated_fp8(A, B, codes, sf, sp, sA, packed, sB, bias, bt, act, pre, M, I,
                                                      K, None))


def gated_bwd(dg, dh=FAKE, pre=FAKE, act=2, codes=FAKE, sf=FAKE, packed=0, dbias=FAKE, M=4, I=256):
    return status(dg, dg.lib.dg_gated_backward_fp8(dh, pre, act, codes, sf, packed, dbias, M, I, None))


def drop(dg, x=FAKE, r=FAKE, xt=1, p=0.1, rng=FAKE, sub=0, out=FAKE, n=100):
    return status(dg, dg.lib.dg_dropout_add(x, r, xt, p, rng, sub, out, n, None))


def drop_bwd(dg, dy=FAKE, xt=1, p=0.1, rng=FAKE, sub=0, codes=FAKE, sf=FAKE, packed=0, dbias=FAKE, M=4, K=256):
    return status(dg, dg.lib.dg_dropout_backward_fp8(dy, xt, p, rng, sub, codes, sf, packed, dbias, M, K, None))


SHAPE, NULL, ALIGN, BIG = "DG_ERR_BAD_SHAPE", "DG_ERR_NULL_POINTER", "DG_ERR_MISALIGNED", "DG_ERR_UNSUPPORTED_SHAPE"


@pytest.mark.parametrize("call", [norm, norm_bwd])
def test_norm_calls_refuse(dg, call):
    for bad in (dict(K=200), dict(M=-1), dict(K=-128), dict(xt=2), dict(wt=-1)):
        assert call(dg, **bad) == SHAPE, bad
    assert call(dg, w=None) == NULL
    for bad in (dict(w=FAKE + 8), dict(h=FAKE + 8), dict(rstd=FAKE + 2), dict(mean=FAKE + 2)):
        assert call(dg, **bad) == ALIGN, bad
    assert call(dg, K=32768 + 128) == BIG and call(dg, M=1 << 33, K=1 << 10) == BIG
    assert call(dg, K=0) == "DG_OK"


def test_norm_refuses(dg):
    for eps in (0.0, -1e-6, float("inf"), float("nan")):
        assert norm(dg, eps=eps) == SHAPE
    for name in ("x", "codes", "sf", "rng"):
        assert norm(dg, **{name: None}) == NULL, name
    for name in ("x", "r", "b", "codes"):
        assert norm(dg, **{name: FAKE + 8}) == ALIGN, name
    assert norm(dg, sf=FAKE + 2) == ALIGN
    assert norm(dg, x=None, w=None, codes=None, sf=None, M=0) == "DG_OK"


def test_norm_backward_refuses(dg):
    for name in ("dy", "h", "mean", "rstd", "dx", "dw"):
        assert norm_bwd(dg, **{name: None}) == NULL, name
    for name in ("dy", "dh", "dx", "dw", "db"):
        assert norm_bwd(dg, **{name: FAKE + 8}) == ALIGN, name
    assert norm_bwd(dg, dw=None, M=0) == NULL


@pytest.mark.parametrize("call", [norm, drop, drop_bwd])
def test_dropout_arguments_refuse(dg, call):
    for p in (-0.1, 1.0, 1 - 2.0 ** -18, 1.5, float("nan"), float("inf")):
        assert call(dg, p=p) == SHAPE, p
    assert call(dg, rng=None) == NULL
    assert call(dg, rng=FAKE + 4) == ALIGN
    empty = dict(n=0) if call is drop else dict(M=0, dbias=None) if call is drop_bwd else dict(M=0)
    assert call(dg, p=0.0, rng=None, **empty) == "DG_OK"
    assert call(dg, p=2.0 ** -18, rng=None, **empty) == "DG_OK"  # rounds to no dropout
    assert call(dg, p=1 - 2.0 ** -16, **empty) == "DG_OK"


def test_dropout_add_refuses(dg):
    assert drop(dg, xt=2) == SHAPE and drop(dg, n=-1) == SHAPE
    assert drop(dg, n=(1 << 40) + 1) == BIG
    for name in ("x", "out"):
        assert drop(dg, **{name: None}) == NULL, name
    for name in ("x", "r", "out"):
        assert drop(dg, **{name: FAKE + 8}) == ALIGN, name


def test_dropout_backward_refuses(dg):
    for bad in (dict(K=200), dict(M=-1), dict(K=-128), dict(xt=2)):
        assert drop_bwd(dg, **bad) == SHAPE, bad
    for name in ("dy", "codes", "sf"):
        assert drop_bwd(dg, **{name: None}) == NULL, name
    for name in ("dy", "codes", "dbias"):
        assert drop_bwd(dg, **{name: FAKE + 8}) == ALIGN, name
    assert drop_bwd(dg, sf=FAKE + 2) == ALIGN
    assert drop_bwd(dg, M=1, K=(1 << 30) + 128) == BIG and drop_bwd(dg, M=1 << 33, K=1 << 10) == BIG


def test_gated_refuses(dg):
    for bad in (dict(I=64), dict(I=-128), dict(M=-1), dict(K=200), dict(K=0), dict(act=5), dict(act=-1), dict(bt=2)):
        assert gated(dg, **bad) == SHAPE, bad
    for name in ("A", "B", "codes", "sf", "sA", "sB"):
        assert gated(dg, **{name: None}) == NULL, name
    for name in ("A", "B", "codes", "bias", "pre"):
        assert gated(dg, **{name: FAKE + 8}) == ALIGN, name
    for name in ("sf", "sA", "sB"):
        assert gated(dg, **{name: FAKE + 2}) == ALIGN, name
    assert gated(dg, M=(1 << 30) + 1) == BIG and gated(dg, I=(1 << 29) + 128) == BIG
    assert gated(dg, K=(1 << 22) + 128) == BIG and gated(dg, I=1 << 21, K=1 << 21) == BIG
    assert gated(dg, M=0) == "DG_OK" and gated(dg, I=0) == "DG_OK"


def test_gated_backward_refuses(dg):
    for bad in (dict(I=200), dict(M=-1), dict(I=-128), dict(act=5)):
        assert gated_bwd(dg, **bad) == SHAPE, bad
    for name in ("dh", "pre", "codes", "sf"):
        assert gated_bwd(dg, **{name: None}) == NULL, name
    for name in ("dh", "pre", "codes", "dbias"):
        assert gated_bwd(dg, **{name: FAKE + 8}) == ALIGN, name
    assert gated_bwd(dg, sf=FAKE + 2) == ALIGN
    assert gated_bwd(dg, M=1, I=(1 << 29) + 128) == BIG and gated_bwd(dg, M=1 << 33, I=1 << 10) == BIG
    assert gated_bwd(dg, M=0, dbias=None) == "DG_OK" and gated_bwd(dg, I=0) == "DG_OK"


def test_binding_refuses(dg):
    x = torch.zeros(4, 256, dtype=torch.bfloat16)
    w = torch.ones(256)
    with pytest.raises(ValueError, match="GPU tensor"):
        dg.layernorm_fp8_1x128(x, w)
    with pytest.raises(ValueError, match=r"\[M, K\]"):
        dg.layernorm_fp8_1x128(x[0], w)
    with pytest.raises(TypeError, match="float32 or torch.bfloat16"):
        dg.layernorm_fp8_1x128(x.half(), w)
    with pytest.raises(ValueError, match=r"\[M, K\]"):
        dg.layernorm_backward(x, x[0], w, w, w)
    with pytest.raises(ValueError, match="GPU tensor"):
        dg.layernorm_backward(x, x, w, w, w)
    with pytest.raises(ValueError, match="GPU tensor"):
        dg.dropout_add(x, 0.1, torch.zeros(2, dtype=torch.int64))
    with pytest.raises(TypeError, match="float32 or torch.bfloat16"):
        dg.dropout_add(x.double(), 0.1, None)
    with pytest.raises(ValueError, match=r"\[M, K\]"):
        dg.dropout_backward_fp8(x[0], 0.1, None)
    with pytest.raises(ValueError, match=r"\[M, I\]"):
        dg.gated_backward_fp8(x[0], x)
    with pytest.raises(ValueError, match="GPU tensor"):
        dg.gated_backward_fp8(x, x)
    a = torch.zeros(4, 128, dtype=torch.uint8)
    with pytest.raises(ValueError, match="GPU tensor"):
        dg.fp8_gemm_nt_gated_fp8(a, a, w, w)
    with pytest.raises(TypeError, match="float8"):
        dg.fp8_gemm_nt_gated_fp8(x, a, w, w)
