"""GPU: an error that another runtime call left in the thread is not reported as a launch's. HIP
keeps the last error until someone asks for it; here an allocation of 2^62 bytes is refused on the
host and nobody asks. The calls after it launch, run once and return."""
import ctypes

import numpy as np
import pytest
import torch

from tests import _block64 as blk

pytestmark = pytest.mark.gpu


def runtime():
    """The HIP runtime that this process has loaded."""
    torch.cuda.init()
    maps = open("/proc/self/maps").read().split()
    return ctypes.CDLL(next(p for p in maps if "libamdhip64" in p))


class Pending:
    """With an error pending in this thread; taken off at the end, before torch looks for its own."""

    def __enter__(self):
        self.hip = runtime()
        torch.cuda.synchronize()
        p = ctypes.c_void_p()
        assert self.hip.hipMalloc(ctypes.byref(p), ctypes.c_size_t(1 << 62)) != 0
        assert self.hip.hipPeekAtLastError() != 0

    def __exit__(self, *exc):
        self.hip.hipGetLastError()


def test_in_place_dropout_runs_once():
    import fp8_block_scaled_dg_amd as m
    x, rng = torch.ones(4096, device="cuda"), torch.tensor([1, 2], device="cuda")
    with Pending():
        m.dropout_add(x, 0.5, rng, out=x)
    assert np.array_equal(x.cpu().numpy(), np.where(blk.kept(0, 4096, 0.5, 1, 2), 2.0, 0.0))


def fp8(*s):
    return torch.full(s, 0x38, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)


def f32(*s):
    return torch.ones(*s, device="cuda")


def bf(*s):
    return torch.ones(*s, dtype=torch.bfloat16, device="cuda")


def test_newer_calls_return():
    import fp8_block_scaled_dg_amd as m
    rng = torch.tensor([1, 2], device="cuda")
    for M in (4, 2000):  # column sums in the same launch, and in a second one
        x, w, mean, rstd, codes, sf, dx = bf(M, 512), bf(512), f32(M), f32(M), fp8(M, 512), f32(M, 4), bf(M, 512)
        dw, db, pre, half, half_sf = f32(512), f32(512), bf(M, 512), bf(M, 256), f32(M, 2)
        a, b, sb, h = fp8(M, 256), fp8(512, 256), f32(4, 2), fp8(M, 256)
        for call in (lambda: m.layernorm_fp8_1x128(x, w, mean=mean, rstd=rstd, codes=codes, sf=sf, dropout_p=0.5, rng=rng),
                     lambda: m.layernorm_backward(x, x, w, mean, rstd, dx=dx, dweight=dw, dbias=db),
                     lambda: m.fp8_gemm_nt_gated_fp8(a, b, half_sf, sb, codes=h, sf=half_sf),
                     lambda: m.gated_backward_fp8(half, pre, codes=codes, sf=sf, dbias=db),
                     lambda: m.dropout_backward_fp8(x, 0.0, rng, codes=codes, sf=sf, dbias=db)):
            with Pending():
                call()
            torch.cuda.synchronize()
        assert torch.all(db == M)


def test_older_calls_return():
    import fp8_block_scaled_dg_amd as m
    for M in (16, 64, 300):  # the rolling, the streaming and the tile kernel
        a, b, c, sa, sb = fp8(M, 2048), fp8(256, 2048), bf(M, 256), f32(M, 16), f32(2, 16)
        with Pending():
            m.fp8_gemm_nt(a, b, c, sa, sb)
        assert torch.all(c == 2048)
        with Pending():
            m.fp8_gemm_nt_bias_act(a, b, c, sa, sb, activation="relu")
        assert torch.all(c == 2048)
    x, w, rstd, dw = bf(300, 256), bf(256), f32(300), torch.empty(256, device="cuda")
    dx, codes, sf = torch.empty_like(x), fp8(300, 256), f32(300, 2)
    with Pending():
        m.quantize_fp8_1x128(x, codes=codes, sf=sf)
    with Pending():
        m.rmsnorm_fp8_1x128(x, w, codes=codes, sf=sf, rstd=rstd)
    with Pending():
        m.rmsnorm_backward(x, x, w, rstd, dx=dx, dweight=dw)
    with Pending():
        m.bias_act_backward_fp8(x, None, None, codes=codes, sf=sf, dbias=dw)
    assert torch.all(dw == 300)
