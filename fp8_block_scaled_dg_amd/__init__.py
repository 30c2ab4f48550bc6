"""Python binding of libdg.so, the MI355X (gfx950) FP8 block-scaled GEMM library.

Argument marshalling only: every call checks dtypes, devices, shapes and contiguity,
then passes raw device pointers and torch's current HIP stream to the C ABI declared
in ``include/dg.h``. All arithmetic runs in the library's HIP kernels; there is no
fallback path. If libdg.so is missing the import fails.

Calls (DeepGEMM project page, aiproducthub.cn, "quick start"; DeepGEMM launch
article, deepseek.csdn.net, section 4.2 "advanced tuning"):

* ``fp8_gemm_nt(a, b, c, a_sf, b_sf)`` and ``fp8_gemm_nn / _tn / _tt`` (other layouts)
* ``m_grouped_fp8_gemm_nt_contiguous(a, b, c, a_sf, b_sf, m_indices)``
* ``m_grouped_fp8_gemm_nt_masked(a, b, c, a_sf, b_sf, masked_m, expected_m=None)``
* ``quantize_fp8_1x128(x, codes=None, sf=None)``: activations -> (A codes, sfA)
* ``m_grouped_fp8_gemm_nt_{contiguous,masked}_swiglu(...)``: Linear1 with a fused
  SwiGLU + requantization epilogue -> (codes, sf) of h = silu(gate) * up
* ``rmsnorm_fp8_1x128(x, weight, eps, residual=...)``: RMS norm of x + residual ->
  (A codes, sfA); ``rmsnorm_backward``: its gradients
* ``fp8_gemm_nt_bias_act(a, b, c, a_sf, b_sf, bias, activation, residual)`` and
  ``fp8_gemm_nt_bias_act_fp8(...)`` -> (codes, sf): the dense GEMM with its epilogue;
  ``bias_act_backward_fp8``: the epilogue's gradients

Operands: ``a``/``b`` are ``torch.float8_e4m3fn`` (``torch.uint8`` holding e4m3fn
codes is accepted too), ``a_sf``/``b_sf`` ``torch.float32``, ``c`` ``torch.bfloat16``
and the index tensors ``torch.int32``, all on the same GPU. An ``a_sf`` of dtype
``torch.int32`` and last dimension ceil(K/512) is the packed UE8M0 layout (one
exponent byte per K-block, four per word) and selects the ``*_ue8m0`` calls.
"""
from __future__ import annotations

import ctypes
import os

import torch  # loaded first: the library then binds to torch's HIP runtime

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libdg.so")

if not os.path.exists(LIB_PATH):
    raise ImportError(
        f"{LIB_PATH} is not built; run `python fp8_block_scaled_dg_amd/build.py` (hipcc, gfx950)")

_vp = ctypes.c_void_p
_i64 = ctypes.c_int64
_i32 = ctypes.c_int32

lib = ctypes.CDLL(LIB_PATH)
lib.dg_build_id.restype = ctypes.c_char_p
lib.dg_build_id.argtypes = []
BUILD_ID = lib.dg_build_id().decode()


def _check_current() -> None:
    """Refuse a libdg.so built from other sources than the ones beside it."""
    from . import build as _build
    try:
        want = _build.source_hash()
    except OSError:  # sources not shipped: nothing to compare with
        return
    if want != BUILD_ID:
        raise ImportError(f"{LIB_PATH} was built from other sources (build id {BUILD_ID}, "
                          f"sources {want}); rebuild it: python fp8_block_scaled_dg_amd/build.py")


_check_current()
lib.dg_fp8_gemm_nt.restype = ctypes.c_int
lib.dg_fp8_gemm_nt.argtypes = [_vp, _vp, _vp, _vp, _vp, _i64, _i64, _i64, _vp]
lib.dg_m_grouped_fp8_gemm_nt_contiguous.restype = ctypes.c_int
lib.dg_m_grouped_fp8_gemm_nt_contiguous.argtypes = [_vp, _vp, _vp, _vp, _vp, _vp, _i64, _i64,
                                                    _i64, _i32, _vp]
lib.dg_m_grouped_fp8_gemm_nt_masked.restype = ctypes.c_int
lib.dg_m_grouped_fp8_gemm_nt_masked.argtypes = [_vp, _vp, _vp, _vp, _vp, _vp, _i32, _i64, _i64,
                                                _i64, _i64, _vp]
lib.dg_status_string.restype = ctypes.c_char_p
lib.dg_status_string.argtypes = [ctypes.c_int]
lib.dg_last_error_detail.restype = ctypes.c_char_p
lib.dg_last_error_detail.argtypes = []
lib.dg_describe_config.restype = ctypes.c_int
lib.dg_describe_config.argtypes = [_i32, _i64, _i64, _i64, _i32, _i64, ctypes.c_char_p, _i64]

lib.dg_fp8_gemm_nt_noalloc.restype = ctypes.c_int
lib.dg_fp8_gemm_nt_noalloc.argtypes = lib.dg_fp8_gemm_nt.argtypes
lib.dg_fp8_gemm_nt_ue8m0.restype = ctypes.c_int
lib.dg_fp8_gemm_nt_ue8m0.argtypes = lib.dg_fp8_gemm_nt.argtypes
lib.dg_m_grouped_fp8_gemm_nt_contiguous_ue8m0.restype = ctypes.c_int
lib.dg_m_grouped_fp8_gemm_nt_contiguous_ue8m0.argtypes = \
    lib.dg_m_grouped_fp8_gemm_nt_contiguous.argtypes
lib.dg_m_grouped_fp8_gemm_nt_masked_ue8m0.restype = ctypes.c_int
lib.dg_m_grouped_fp8_gemm_nt_masked_ue8m0.argtypes = lib.dg_m_grouped_fp8_gemm_nt_masked.argtypes
lib.dg_m_grouped_fp8_gemm_nt_contiguous_swiglu.restype = ctypes.c_int
lib.dg_m_grouped_fp8_gemm_nt_contiguous_swiglu.argtypes = [_vp, _vp, _vp, _vp, _vp, _vp, _vp,
                                                          _i64, _i64, _i64, _i32, _vp]
lib.dg_m_grouped_fp8_gemm_nt_masked_swiglu.restype = ctypes.c_int
lib.dg_m_grouped_fp8_gemm_nt_masked_swiglu.argtypes = [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _i32,
                                                      _i64, _i64, _i64, _vp]
for _name in ("dg_fp8_gemm_nn", "dg_fp8_gemm_tn", "dg_fp8_gemm_tt"):
    getattr(lib, _name).restype = ctypes.c_int
    getattr(lib, _name).argtypes = lib.dg_fp8_gemm_nt.argtypes
lib.dg_quantize_fp8_1x128.restype = ctypes.c_int
lib.dg_quantize_fp8_1x128.argtypes = [_vp, _i32, _vp, _vp, _i64, _i64, _vp]

lib.dg_rmsnorm_fp8_1x128.restype = ctypes.c_int
lib.dg_rmsnorm_fp8_1x128.argtypes = [_vp, _vp, _i32, _vp, _i32, ctypes.c_float, _vp, _vp, _vp, _vp,
                                     _i32, _i64, _i64, _vp]
lib.dg_rmsnorm_backward.restype = ctypes.c_int
lib.dg_rmsnorm_backward.argtypes = [_vp, _vp, _vp, _i32, _vp, _i32, _vp, _vp, _vp, _i64, _i64, _vp]
lib.dg_fp8_gemm_nt_bias_act.restype = ctypes.c_int
lib.dg_fp8_gemm_nt_bias_act.argtypes = [_vp, _vp, _vp, _vp, _i32, _vp, _vp, _i32, _i32, _vp, _vp,
                                        _i64, _i64, _i64, _vp]
lib.dg_fp8_gemm_nt_bias_act_fp8.restype = ctypes.c_int
lib.dg_fp8_gemm_nt_bias_act_fp8.argtypes = [_vp, _vp, _vp, _vp, _i32, _vp, _i32, _vp, _vp, _i32,
                                            _i32, _vp, _i64, _i64, _i64, _vp]
lib.dg_bias_act_backward_fp8.restype = ctypes.c_int
lib.dg_bias_act_backward_fp8.argtypes = [_vp, _vp, _i32, _vp, _vp, _i32, _vp, _i64, _i64, _vp]

lib.dg_release_workspaces.restype = ctypes.c_int
lib.dg_release_workspaces.argtypes = []
lib.dg_num_configs.restype = _i32
lib.dg_num_configs.argtypes = []
lib.dg_config_name.restype = ctypes.c_char_p
lib.dg_config_name.argtypes = [_i32]

KIND_DENSE, KIND_CONTIGUOUS, KIND_MASKED = 0, 1, 2
DTYPE_F32, DTYPE_BF16 = 0, 1
ACTIVATIONS = {None: 0, "none": 0, "relu": 1, "silu": 2, "gelu": 3, "gelu_tanh": 4}
BLOCK = 128


class DGError(RuntimeError):
    def __init__(self, status: int):
        self.status = status
        name = lib.dg_status_string(status).decode()
        detail = lib.dg_last_error_detail().decode()
        super().__init__(f"{name}: {detail}" if detail else name)


def check(status: int) -> None:
    if status != 0:
        raise DGError(status)


def _fp8(t: torch.Tensor, name: str) -> torch.Tensor:
    if t.dtype not in (torch.float8_e4m3fn, torch.uint8):
        raise TypeError(f"{name} must be torch.float8_e4m3fn (or uint8 codes), got {t.dtype}")
    return t


def _need(t: torch.Tensor, name: str, dtype: torch.dtype, shape: tuple, device) -> None:
    # one combined test on the common path; the specific error only on failure
    if t.dtype != dtype or t.shape != shape or t.device != device or not t.is_contiguous():
        if t.dtype != dtype:
            raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
        if tuple(t.shape) != tuple(shape):
            raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
        _dev(t, name, device)


def _dev(t: torch.Tensor, name: str, device) -> None:
    if not t.is_cuda:
        raise ValueError(f"{name} must be a GPU tensor")
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


_current_device = torch.cuda.current_device
_raw_stream = torch._C._cuda_getCurrentRawStream


def _run(dev, fn, *args) -> None:
    """fn(*args, stream): the library call on torch's current stream of `dev`, with
    `dev` the current device (the library keeps its workspace per device and stream).
    The device is switched only when it is not current already. Raises DGError on a
    nonzero status."""
    idx = dev.index
    if _current_device() == idx:
        status = fn(*args, _raw_stream(idx))
    else:
        with torch.cuda.device(idx):
            status = fn(*args, _raw_stream(idx))
    if status:
        raise DGError(status)


def _a_sf_layout(a_sf, lead: tuple, K: int, dev):
    """(packed?, expected shape) of a_sf: torch.float32 [..., K/128], or torch.int32
    [..., ceil(K/512)] holding packed UE8M0 bytes (one per K-block, 4 per word)."""
    if a_sf.dtype == torch.int32:
        shape = lead + ((K // BLOCK + 3) // 4,)
        _need(a_sf, "a_sf", torch.int32, shape, dev)
        return True
    _need(a_sf, "a_sf", torch.float32, lead + (K // BLOCK,), dev)
    return False


def fp8_gemm_nt(a, b, c, a_sf, b_sf) -> None:
    """c[M][N] (bf16) = block-scaled a[M][K] x b[N][K]^T; writes c in place. a_sf is
    fp32 [M, K/128], or int32 [M, ceil(K/512)] in the packed UE8M0 layout."""
    _fp8(a, "a"), _fp8(b, "b")
    if a.dim() != 2 or b.dim() != 2:
        raise ValueError("a and b must be 2-D")
    M, K = a.shape
    N = b.shape[0]
    dev = a.device
    _dev(a, "a", dev)
    _need(b, "b", b.dtype, (N, K), dev)
    _need(c, "c", torch.bfloat16, (M, N), dev)
    packed = _a_sf_layout(a_sf, (M,), K, dev)
    _need(b_sf, "b_sf", torch.float32, ((N + BLOCK - 1) // BLOCK, K // BLOCK), dev)
    fn = lib.dg_fp8_gemm_nt_ue8m0 if packed else lib.dg_fp8_gemm_nt
    _run(dev, fn, a.data_ptr(), b.data_ptr(), c.data_ptr(), a_sf.data_ptr(), b_sf.data_ptr(),
         M, N, K)


def _fp8_gemm_layout(layout: str, a, b, c, a_sf, b_sf) -> None:
    _fp8(a, "a"), _fp8(b, "b")
    if a.dim() != 2 or b.dim() != 2:
        raise ValueError("a and b must be 2-D")
    M, K = (a.shape[1], a.shape[0]) if layout[0] == "t" else tuple(a.shape)
    N = b.shape[1] if layout[1] == "n" else b.shape[0]
    dev = a.device
    _dev(a, "a", dev)
    _need(b, "b", b.dtype, (K, N) if layout[1] == "n" else (N, K), dev)
    _need(c, "c", torch.bfloat16, (M, N), dev)
    _need(a_sf, "a_sf", torch.float32, (M, K // BLOCK), dev)
    _need(b_sf, "b_sf", torch.float32, ((N + BLOCK - 1) // BLOCK, K // BLOCK), dev)
    fn = getattr(lib, "dg_fp8_gemm_" + layout)
    _run(dev, fn, a.data_ptr(), b.data_ptr(), c.data_ptr(), a_sf.data_ptr(), b_sf.data_ptr(),
         M, N, K)


def fp8_gemm_nn(a, b, c, a_sf, b_sf) -> None:
    """c [M][N] = a [M][K] x b [K][N] (block-scaled; scales as for fp8_gemm_nt)."""
    _fp8_gemm_layout("nn", a, b, c, a_sf, b_sf)


def fp8_gemm_tn(a, b, c, a_sf, b_sf) -> None:
    """c [M][N] = a [K][M]^T x b [K][N]."""
    _fp8_gemm_layout("tn", a, b, c, a_sf, b_sf)


def fp8_gemm_tt(a, b, c, a_sf, b_sf) -> None:
    """c [M][N] = a [K][M]^T x b [N][K]^T."""
    _fp8_gemm_layout("tt", a, b, c, a_sf, b_sf)


def m_grouped_fp8_gemm_nt_contiguous(a, b, c, a_sf, b_sf, m_indices) -> None:
    """Contiguous MoE layout: row r of a uses expert m_indices[r]'s b (-1 = pad row,
    left untouched in c)."""
    _fp8(a, "a"), _fp8(b, "b")
    if a.dim() != 2 or b.dim() != 3:
        raise ValueError("a must be [M_total, K] and b [G, N, K]")
    M, K = a.shape
    G, N = b.shape[0], b.shape[1]
    dev = a.device
    _dev(a, "a", dev)
    _need(b, "b", b.dtype, (G, N, K), dev)
    _need(c, "c", torch.bfloat16, (M, N), dev)
    packed = _a_sf_layout(a_sf, (M,), K, dev)
    _need(b_sf, "b_sf", torch.float32, (G, (N + BLOCK - 1) // BLOCK, K // BLOCK), dev)
    _need(m_indices, "m_indices", torch.int32, (M,), dev)
    fn = (lib.dg_m_grouped_fp8_gemm_nt_contiguous_ue8m0 if packed
          else lib.dg_m_grouped_fp8_gemm_nt_contiguous)
    _run(dev, fn, a.data_ptr(), b.data_ptr(), c.data_ptr(), a_sf.data_ptr(), b_sf.data_ptr(),
         m_indices.data_ptr(), M, N, K, G)


def m_grouped_fp8_gemm_nt_masked(a, b, c, a_sf, b_sf, masked_m, expected_m=None) -> None:
    """Masked MoE layout: expert e computes its first masked_m[e] rows of a[e]; the
    other rows of c[e] are left untouched."""
    _fp8(a, "a"), _fp8(b, "b")
    if a.dim() != 3 or b.dim() != 3:
        raise ValueError("a must be [G, M_max, K] and b [G, N, K]")
    G, M_max, K = a.shape
    N = b.shape[1]
    dev = a.device
    _dev(a, "a", dev)
    _need(b, "b", b.dtype, (G, N, K), dev)
    _need(c, "c", torch.bfloat16, (G, M_max, N), dev)
    packed = _a_sf_layout(a_sf, (G, M_max), K, dev)
    _need(b_sf, "b_sf", torch.float32, (G, (N + BLOCK - 1) // BLOCK, K // BLOCK), dev)
    _need(masked_m, "masked_m", torch.int32, (G,), dev)
    em = int(expected_m) if expected_m is not None else 0
    fn = lib.dg_m_grouped_fp8_gemm_nt_masked_ue8m0 if packed else lib.dg_m_grouped_fp8_gemm_nt_masked
    _run(dev, fn, a.data_ptr(), b.data_ptr(), c.data_ptr(), a_sf.data_ptr(), b_sf.data_ptr(),
         masked_m.data_ptr(), G, M_max, N, K, em)


def _swiglu_outputs(lead: tuple, I: int, codes, sf, dev):
    if codes is None:
        codes = torch.empty(lead + (I,), dtype=torch.float8_e4m3fn, device=dev)
    if sf is None:
        sf = torch.empty(lead + (I // BLOCK,), dtype=torch.float32, device=dev)
    _fp8(codes, "codes")
    _need(codes, "codes", codes.dtype, lead + (I,), dev)
    _need(sf, "sf", torch.float32, lead + (I // BLOCK,), dev)
    return codes, sf


def m_grouped_fp8_gemm_nt_contiguous_swiglu(a, b, a_sf, b_sf, m_indices, codes=None, sf=None):
    """Contiguous MoE Linear1 with the fused SwiGLU + 1x128 requantization epilogue.
    b is [G, 2I, K] (gate rows, then up rows); returns (codes [M_total, I] e4m3fn,
    sf [M_total, I/128] fp32) of h = silu(gate) * up, written into the given tensors
    when passed. Pad rows are not written."""
    _fp8(a, "a"), _fp8(b, "b")
    if a.dim() != 2 or b.dim() != 3 or b.shape[1] % 2:
        raise ValueError("a must be [M_total, K] and b [G, 2I, K]")
    M, K = a.shape
    G, N2 = b.shape[0], b.shape[1]
    I = N2 // 2
    dev = a.device
    _dev(a, "a", dev)
    _need(b, "b", b.dtype, (G, N2, K), dev)
    _need(a_sf, "a_sf", torch.float32, (M, K // BLOCK), dev)
    _need(b_sf, "b_sf", torch.float32, (G, N2 // BLOCK, K // BLOCK), dev)
    _need(m_indices, "m_indices", torch.int32, (M,), dev)
    codes, sf = _swiglu_outputs((M,), I, codes, sf, dev)
    _run(dev, lib.dg_m_grouped_fp8_gemm_nt_contiguous_swiglu, a.data_ptr(), b.data_ptr(),
         codes.data_ptr(), sf.data_ptr(), a_sf.data_ptr(), b_sf.data_ptr(), m_indices.data_ptr(),
         M, I, K, G)
    return codes, sf


def m_grouped_fp8_gemm_nt_masked_swiglu(a, b, a_sf, b_sf, masked_m, codes=None, sf=None):
    """Masked MoE Linear1 with the fused SwiGLU + 1x128 requantization epilogue:
    returns (codes [G, M_max, I], sf [G, M_max, I/128]); rows >= masked_m[e] are not
    written."""
    _fp8(a, "a"), _fp8(b, "b")
    if a.dim() != 3 or b.dim() != 3 or b.shape[1] % 2:
        raise ValueError("a must be [G, M_max, K] and b [G, 2I, K]")
    G, M_max, K = a.shape
    N2 = b.shape[1]
    I = N2 // 2
    dev = a.device
    _dev(a, "a", dev)
    _need(b, "b", b.dtype, (G, N2, K), dev)
    _need(a_sf, "a_sf", torch.float32, (G, M_max, K // BLOCK), dev)
    _need(b_sf, "b_sf", torch.float32, (G, N2 // BLOCK, K // BLOCK), dev)
    _need(masked_m, "masked_m", torch.int32, (G,), dev)
    codes, sf = _swiglu_outputs((G, M_max), I, codes, sf, dev)
    _run(dev, lib.dg_m_grouped_fp8_gemm_nt_masked_swiglu, a.data_ptr(), b.data_ptr(),
         codes.data_ptr(), sf.data_ptr(), a_sf.data_ptr(), b_sf.data_ptr(), masked_m.data_ptr(),
         G, M_max, I, K)
    return codes, sf


def quantize_fp8_1x128(x, codes=None, sf=None):
    """Per-token 1x128 quantization of x [M, K] (float32 or bfloat16): returns
    (codes [M, K] torch.float8_e4m3fn, sf [M, K/128] torch.float32), written into the
    given tensors when passed (new tensors otherwise)."""
    if x.dim() != 2:
        raise ValueError("x must be [M, K]")
    if x.dtype == torch.float32:
        dtype = DTYPE_F32
    elif x.dtype == torch.bfloat16:
        dtype = DTYPE_BF16
    else:
        raise TypeError(f"x must be torch.float32 or torch.bfloat16, got {x.dtype}")
    M, K = x.shape
    dev = x.device
    _dev(x, "x", dev)
    if codes is None:
        codes = torch.empty((M, K), dtype=torch.float8_e4m3fn, device=dev)
    if sf is None:
        sf = torch.empty((M, K // BLOCK), dtype=torch.float32, device=dev)
    _fp8(codes, "codes")
    _need(codes, "codes", codes.dtype, (M, K), dev)
    _need(sf, "sf", torch.float32, (M, K // BLOCK), dev)
    _run(dev, lib.dg_quantize_fp8_1x128, x.data_ptr(), dtype, codes.data_ptr(), sf.data_ptr(),
         M, K)
    return codes, sf


_DTYPES = {torch.float32: DTYPE_F32, torch.bfloat16: DTYPE_BF16}
_get_device = torch._C._cuda_getDevice


def _float_type(t: torch.Tensor, name: str) -> int:
    d = _DTYPES.get(t.dtype)
    if d is None:
        raise TypeError(f"{name} must be torch.float32 or torch.bfloat16, got {t.dtype}")
    return d


def _act(activation) -> int:
    code = ACTIVATIONS.get(activation)
    if code is None:
        raise ValueError(f"activation must be one of {list(ACTIVATIONS)}, got {activation!r}")
    return code


def _ptr(t: torch.Tensor, name: str, dtype: torch.dtype, shape, x: torch.Tensor, index: int) -> int:
    """t's address, once it has this dtype and shape, is contiguous and lies on the GPU
    `index` of x (the test of _need in its quickest form; a call checks up to seven tensors)."""
    if (t.dtype is not dtype or t.get_device() != index or t.shape != shape
            or not t.is_contiguous()):
        _need(t, name, dtype, tuple(shape), x.device)
    return t.data_ptr()


def _first(x: torch.Tensor, name: str) -> int:
    """The GPU index of a call's first tensor, which has to be contiguous."""
    index = x.get_device()
    if index < 0 or not x.is_contiguous():
        _dev(x, name, x.device)
    return index


def _launch(index: int, fn, *args) -> None:
    """_run for a GPU index; a call's tensors exist, so HIP is initialised."""
    if _get_device() == index:
        status = fn(*args, _raw_stream(index))
    else:
        with torch.cuda.device(index):
            status = fn(*args, _raw_stream(index))
    if status:
        raise DGError(status)


def _fp8_outputs(M: int, N: int, codes, sf, ue8m0: bool, x: torch.Tensor, index: int):
    """(codes, codes pointer, sf, sf pointer, packed?) of an FP8 output [M, N]: new tensors
    where none is passed. The dtype of a passed sf (float32, or int32 for packed UE8M0) says
    its form."""
    if codes is None:
        codes = torch.empty((M, N), dtype=torch.float8_e4m3fn, device=x.device)
        codes_ptr = codes.data_ptr()
    else:
        _fp8(codes, "codes")
        codes_ptr = _ptr(codes, "codes", codes.dtype, (M, N), x, index)
    if sf is None:
        sf = (torch.empty((M, (N // BLOCK + 3) // 4), dtype=torch.int32, device=x.device) if ue8m0
              else torch.empty((M, N // BLOCK), dtype=torch.float32, device=x.device))
        return codes, codes_ptr, sf, sf.data_ptr(), ue8m0
    if sf.dtype is torch.int32:
        return codes, codes_ptr, sf, _ptr(sf, "sf", torch.int32, (M, (N // BLOCK + 3) // 4), x, index), True
    return codes, codes_ptr, sf, _ptr(sf, "sf", torch.float32, (M, N // BLOCK), x, index), False


def rmsnorm_fp8_1x128(x, weight, eps=1e-6, residual=None, h=None, rstd=None, codes=None, sf=None,
                      ue8m0=False):
    """RMS norm of x + residual ([M, K] float32 or bfloat16) with weight [K], quantized per
    1x128 block: returns (codes [M, K] e4m3fn, sf), the a and a_sf of the GEMM calls. sf is
    fp32 [M, K/128], or int32 [M, ceil(K/512)] packed UE8M0 (ue8m0=True, or a passed sf of
    that dtype). h, when passed, receives x + residual (it may be x or residual itself),
    rstd (fp32 [M]) 1 / rms; rmsnorm_backward takes both."""
    if x.dim() != 2:
        raise ValueError("x must be [M, K]")
    dtype, w_dtype = _float_type(x, "x"), _float_type(weight, "weight")
    M, K = shape = x.shape
    dev = _first(x, "x")
    w = _ptr(weight, "weight", weight.dtype, (K,), x, dev)
    r = None if residual is None else _ptr(residual, "residual", x.dtype, shape, x, dev)
    hp = None if h is None else _ptr(h, "h", x.dtype, shape, x, dev)
    rs = None if rstd is None else _ptr(rstd, "rstd", torch.float32, (M,), x, dev)
    codes, cp, sf, sp, packed = _fp8_outputs(M, K, codes, sf, ue8m0, x, dev)
    _launch(dev, lib.dg_rmsnorm_fp8_1x128, x.data_ptr(), r, dtype, w, w_dtype, eps, hp, rs, cp, sp,
            packed, M, K)
    return codes, sf


def rmsnorm_backward(dy, h, weight, rstd, dh=None, dx=None, dweight=None):
    """Gradients of rmsnorm_fp8_1x128 (the quantization taken as the identity), from the h
    and rstd it stored: returns (dx [M, K] of h's dtype, dweight [K] float32). dh, the
    gradient that reaches h along the residual stream, is added to dx; dx is the gradient
    of x and of residual alike, and may be dy, dh or h itself."""
    if h.dim() != 2:
        raise ValueError("h must be [M, K]")
    dtype, w_dtype = _float_type(h, "h"), _float_type(weight, "weight")
    M, K = shape = h.shape
    dev = _first(h, "h")
    g = _ptr(dy, "dy", h.dtype, shape, h, dev)
    w = _ptr(weight, "weight", weight.dtype, (K,), h, dev)
    rs = _ptr(rstd, "rstd", torch.float32, (M,), h, dev)
    r = None if dh is None else _ptr(dh, "dh", h.dtype, shape, h, dev)
    if dx is None:
        dx = torch.empty_like(h)
    if dweight is None:
        dweight = torch.empty((K,), dtype=torch.float32, device=h.device)
    _launch(dev, lib.dg_rmsnorm_backward, g, r, h.data_ptr(), dtype, w, w_dtype, rs,
            _ptr(dx, "dx", h.dtype, shape, h, dev), _ptr(dweight, "dweight", torch.float32, (K,), h, dev),
            M, K)
    return dx, dweight


def _bias_act_operands(a, b, a_sf, b_sf, bias, pre):
    """Checks what the two epilogue GEMMs share: (M, N, K, GPU index, a, b, a_sf, packed?,
    b_sf, bias, bias dtype, pre), tensors as addresses."""
    _fp8(a, "a"), _fp8(b, "b")
    if a.dim() != 2 or b.dim() != 2:
        raise ValueError("a and b must be 2-D")
    M, K = a.shape
    N = b.shape[0]
    dev = _first(a, "a")
    bp = _ptr(b, "b", b.dtype, (N, K), a, dev)
    KB = K // BLOCK
    packed = a_sf.dtype is torch.int32
    ap = (_ptr(a_sf, "a_sf", torch.int32, (M, (KB + 3) // 4), a, dev) if packed
          else _ptr(a_sf, "a_sf", torch.float32, (M, KB), a, dev))
    sp = _ptr(b_sf, "b_sf", torch.float32, ((N + BLOCK - 1) // BLOCK, KB), a, dev)
    bias_ptr, bias_dtype = None, 0
    if bias is not None:
        bias_dtype = _float_type(bias, "bias")
        bias_ptr = _ptr(bias, "bias", bias.dtype, (N,), a, dev)
    pre_ptr = None if pre is None else _ptr(pre, "pre", torch.bfloat16, (M, N), a, dev)
    return M, N, K, dev, a.data_ptr(), bp, ap, packed, sp, bias_ptr, bias_dtype, pre_ptr


def fp8_gemm_nt_bias_act(a, b, c, a_sf, b_sf, bias=None, activation=None, residual=None,
                         pre=None) -> None:
    """c [M, N] (bf16) = activation(a x b^T + bias) + residual, rounded once; writes c in
    place. a, b and the scales as for fp8_gemm_nt; bias [N] float32 or bfloat16; activation
    None, "relu", "silu", "gelu" or "gelu_tanh"; residual [M, N] bf16 (c itself is allowed);
    pre, when passed, receives a x b^T + bias (bf16 [M, N], for bias_act_backward_fp8)."""
    M, N, K, dev, ap, bp, sa, packed, sb, bias_ptr, bias_dtype, pre_ptr = \
        _bias_act_operands(a, b, a_sf, b_sf, bias, pre)
    cp = _ptr(c, "c", torch.bfloat16, (M, N), a, dev)
    r = None if residual is None else _ptr(residual, "residual", torch.bfloat16, (M, N), a, dev)
    _launch(dev, lib.dg_fp8_gemm_nt_bias_act, ap, bp, cp, sa, packed, sb, bias_ptr, bias_dtype,
            _act(activation), r, pre_ptr, M, N, K)


def fp8_gemm_nt_bias_act_fp8(a, b, a_sf, b_sf, bias=None, activation=None, pre=None, codes=None,
                             sf=None, ue8m0=False):
    """activation(a x b^T + bias) quantized per 1x128 block: returns (codes [M, N] e4m3fn,
    sf), the next GEMM's a and a_sf (sf as in rmsnorm_fp8_1x128). N % 128 == 0; the other
    arguments as for fp8_gemm_nt_bias_act."""
    M, N, K, dev, ap, bp, sa, packed, sb, bias_ptr, bias_dtype, pre_ptr = \
        _bias_act_operands(a, b, a_sf, b_sf, bias, pre)
    codes, cp, sf, sp, sf_packed = _fp8_outputs(M, N, codes, sf, ue8m0, a, dev)
    _launch(dev, lib.dg_fp8_gemm_nt_bias_act_fp8, ap, bp, cp, sp, sf_packed, sa, packed, sb, bias_ptr,
            bias_dtype, _act(activation), pre_ptr, M, N, K)
    return codes, sf


def bias_act_backward_fp8(dc, pre=None, activation=None, codes=None, sf=None, dbias=None,
                          need_dbias=True, ue8m0=False):
    """Backward of the bias + activation epilogue: p = dc * activation'(pre) (dc, pre bf16
    [M, N]; pre may be None without an activation), returned as (codes, sf, dbias): p
    quantized per 1x128 block and dbias [N] float32 = p summed over rows (None with
    need_dbias=False). The input's gradient is then fp8_gemm_nn(codes, b, da, sf,
    b_sf.t().contiguous()) with the forward call's b."""
    if dc.dim() != 2:
        raise ValueError("dc must be [M, N]")
    M, N = shape = dc.shape
    dev = _first(dc, "dc")
    d = _ptr(dc, "dc", torch.bfloat16, shape, dc, dev)
    act = _act(activation)
    z = None if pre is None else _ptr(pre, "pre", torch.bfloat16, shape, dc, dev)
    codes, cp, sf, sp, packed = _fp8_outputs(M, N, codes, sf, ue8m0, dc, dev)
    if dbias is None and need_dbias:
        dbias = torch.empty((N,), dtype=torch.float32, device=dc.device)
    db = None if dbias is None else _ptr(dbias, "dbias", torch.float32, (N,), dc, dev)
    _launch(dev, lib.dg_bias_act_backward_fp8, d, z, act, cp, sp, packed, db, M, N)
    return codes, sf, dbias


def release_workspaces() -> None:
    """Free the library's own device buffers (split-K partials and counters, transposed
    operand copies) after the devices holding them go idle. No HIP graph holding a
    library call may be replayed afterwards."""
    check(lib.dg_release_workspaces())


def describe_config(kind: int, M: int, N: int, K: int, G: int = 1, expected_m: int = 0) -> str:
    buf = ctypes.create_string_buffer(128)
    check(lib.dg_describe_config(kind, M, N, K, G, expected_m, buf, 128))
    return buf.value.decode()


def config_names() -> list[str]:
    return [lib.dg_config_name(i).decode() for i in range(lib.dg_num_configs())]


__all__ = ["config_names", "fp8_gemm_nt", "fp8_gemm_nn", "fp8_gemm_tn", "fp8_gemm_tt", "m_grouped_fp8_gemm_nt_contiguous", "m_grouped_fp8_gemm_nt_masked",
           "m_grouped_fp8_gemm_nt_contiguous_swiglu", "m_grouped_fp8_gemm_nt_masked_swiglu",
           "quantize_fp8_1x128", "rmsnorm_fp8_1x128", "rmsnorm_backward", "fp8_gemm_nt_bias_act",
           "fp8_gemm_nt_bias_act_fp8", "bias_act_backward_fp8", "ACTIVATIONS", "describe_config", "release_workspaces", "BUILD_ID", "DGError", "lib", "LIB_PATH"]
