"""GPU: the native marshalling (csrc/marshal.cpp) calls the library once, whatever it reports.
A call that writes in place (dropout_add(x, out=x), a layer norm's h or dx in place of its input)
would compute on its own output if it were made again."""
import ctypes

import pytest
import torch

pytestmark = pytest.mark.gpu
BF = torch.bfloat16
CALLS = ("dg_layernorm_fp8_1x128", "dg_layernorm_backward", "dg_fp8_gemm_nt_gated_fp8", "dg_gated_backward_fp8",
         "dg_dropout_add", "dg_dropout_backward_fp8")


def dg():
    import fp8_block_scaled_dg_amd as m
    return m


def calls():
    """Each call with arguments that the native checks take, in place where there is such a form."""
    m = dg()
    bf = lambda *s: torch.ones(*s, dtype=BF, device="cuda")  # noqa: E731
    f32 = lambda *s: torch.ones(*s, device="cuda")  # noqa: E731
    fp8 = lambda *s: torch.zeros(*s, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)  # noqa: E731
    rng = torch.tensor([1, 2], device="cuda")
    x, dy = bf(4, 256), bf(4, 256)
    return (lambda: m.layernorm_fp8_1x128(x, bf(256), h=x, dropout_p=0.5, rng=rng),
            lambda: m.layernorm_backward(dy, bf(4, 256), bf(256), f32(4), f32(4), dx=dy),
            lambda: m.fp8_gemm_nt_gated_fp8(fp8(4, 256), fp8(256, 256), f32(4, 2), f32(2, 2)),
            lambda: m.gated_backward_fp8(bf(4, 128), bf(4, 256)),
            lambda: m.dropout_add(x, 0.5, rng, out=x),
            lambda: m.dropout_backward_fp8(x, 0.5, rng))


@pytest.mark.parametrize("status", [6, 7])
def test_a_failed_call_is_made_once(status, monkeypatch):
    m = dg()
    native, python = [], []

    def stub(i):
        def body(*args):
            native.append(i)
            return status
        return body

    real = [ctypes.cast(getattr(m.lib, name), ctypes.c_void_p).value for name in CALLS]
    stubs = []
    for i, name in enumerate(CALLS):
        stubs.append(ctypes.CFUNCTYPE(ctypes.c_int, *getattr(m.lib, name).argtypes)(stub(i)))
        monkeypatch.setattr(m.lib, name, lambda *args, i=i: python.append(i) or status)
    try:
        m._marshal.bind(*(ctypes.cast(s, ctypes.c_void_p).value for s in stubs), m.check)
        for i, call in enumerate(calls()):
            native.clear()
            with pytest.raises(m.DGError) as e:
                call()
            assert e.value.status == status
            assert native == [i] and not python, CALLS[i]
    finally:
        m._marshal.bind(*real, m.check)


def test_calls_return_what_they_made():
    for call, n in zip(calls(), (2, 3, 2, 3, 1, 3)):
        r = call()
        torch.cuda.synchronize()
        assert len(r) == n if n > 1 else isinstance(r, torch.Tensor)


def test_refusals_name_their_cause():
    m = dg()
    x, rng = torch.ones(16, device="cuda"), torch.tensor([1, 2], device="cuda")
    for bad, match in ((lambda: m.dropout_add(x, 1.0, rng), "dropout_p"), (lambda: m.dropout_add(x, 0.5, None), "NULL rng"),
                       (lambda: m.dropout_add(torch.ones(17, device="cuda")[1:], 0.5, rng), "16-byte aligned")):
        with pytest.raises(m.DGError, match=match):
            bad()
