"""Thin Python binding of libnvfp4.so (include/nvfp4.h).

Argument marshalling only: every step of the method runs in the library's
CUDA kernels.  PyTorch provides device memory and the current stream.  There
is no CPU fallback: if the shared library is missing or the device is not a
B200 (sm_100), calls raise.

The raw C functions are available as ``lib().<name>`` (ctypes), with the same
names and arguments as the header; the wrappers below allocate outputs with
torch and pass device pointers plus ``torch.cuda.current_stream()``.
"""
from __future__ import annotations

import ctypes
import functools
import os

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libnvfp4.so")

OK, ERR_INVALID_ARG, ERR_UNSUPPORTED, ERR_CUDA, ERR_TIMEOUT, ERR_DEVICE_INDEX = range(6)
DT = {torch.float32: 0, torch.float16: 1, torch.bfloat16: 2}
LAYOUT = {"linear": 0, "swizzled": 1}
MODE = {"nvfp4": 0, "mxfp8": 1, "mxfp4": 2}

# (name, restype, argtypes) of every symbol declared in include/nvfp4.h
_P, _I64, _I, _SZ = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_size_t


class AmaxItem(ctypes.Structure):
    """nvfp4_amax_item"""
    _fields_ = [("x", _P), ("n", _I64), ("g_out", _P)]


class QuantizeItem(ctypes.Structure):
    """nvfp4_quantize_item (the layout enum is a C int)"""
    _fields_ = [("x", _P), ("rows", _I64), ("K", _I64), ("g", _P), ("codes", _P), ("scales", _P),
                ("layout", _I)]


class KvCacheArgs(ctypes.Structure):
    """nvfp4_kv_cache"""
    _fields_ = [("mode", _I), ("num_pages", _I64), ("page_size", _I64), ("heads", _I64), ("D", _I64),
                ("k_codes", _P), ("k_scales", _P), ("v_codes", _P), ("v_scales", _P), ("g_k", _P), ("g_v", _P)]


SIGNATURES = [
    ("nvfp4_status_string", ctypes.c_char_p, [_I]),
    ("nvfp4_last_error_message", ctypes.c_char_p, []),
    ("nvfp4_check_device_errors", _I, [_P]),
    ("nvfp4_scale_bytes", _SZ, [_I64, _I64, _I]),
    ("nvfp4_amax", _I, [_P, _I, _I64, _P, _P]),
    ("nvfp4_amax_multi", _I, [ctypes.POINTER(AmaxItem), _I, _I, _P]),
    ("nvfp4_quantize", _I, [_P, _I, _I64, _I64, _P, _P, _P, _I, _P]),
    ("nvfp4_quantize_multi", _I, [ctypes.POINTER(QuantizeItem), _I, _I, _P]),
    ("nvfp4_quantize_columnwise", _I, [_P, _I, _I64, _I64, _P, _P, _P, _I, _P]),
    ("nvfp4_dequantize", _I, [_P, _P, _I, _I64, _I64, _P, _P, _I, _P]),
    ("nvfp4_quantize_sr", _I, [_P, _I, _I64, _I64, _P, ctypes.c_uint64, _P, _P, _I, _P]),
    ("nvfp4_quantize_columnwise_sr", _I, [_P, _I, _I64, _I64, _P, ctypes.c_uint64, _P, _P, _I, _P]),
    ("mxfp8_quantize", _I, [_P, _I, _I64, _I64, _P, _P, _I, _P]),
    ("mxfp8_dequantize", _I, [_P, _P, _I, _I64, _I64, _P, _I, _P]),
    ("mxfp4_quantize", _I, [_P, _I, _I64, _I64, _P, _P, _I, _P]),
    ("mxfp4_dequantize", _I, [_P, _P, _I, _I64, _I64, _P, _I, _P]),
    ("nvfp4_swizzle_scales", _I, [_P, _I64, _I64, _P, _P]),
    ("qqmm", _I, [_I, _I64, _I64, _I64, _P, _P, _P, _P, _P, _P, _P, _I, _P]),
    ("qmv", _I, [_P, _I, _P, _P, _P, _P, _I64, _I64, _I64, _P, _P]),
    ("qmv_pdl", _I, [_P, _I, _P, _P, _P, _P, _I64, _I64, _I64, _P, _P]),
    ("qmv_mx", _I, [_I, _P, _I, _P, _P, _I64, _I64, _I64, _P, _P]),
    ("gather_qmm", _I, [_P, _P, _P, _P, _P, _I64, _I64, _I64, _I64, _I64, _P, _P, _SZ, _P]),
    ("gather_qmm_kn", _I, [_P, _P, _P, _P, _P, _I64, _I64, _I64, _I64, _I64, _P, _P, _SZ, _P]),
    ("gather_qmm_workspace_size", _SZ, [_I64, _I64, _I64]),
    ("gather_qmm_staged_workspace_size", _SZ, [_I64, _I64, _I64, _I64]),
    ("gather_qmm_noalloc", _I, [_P, _P, _P, _P, _P, _I64, _I64, _I64, _I64, _I64, _P, _P]),
    ("rms_norm", _I, [_P, _P, _P, _I, _I64, _I64, ctypes.c_double, _P, _P, _P, _P]),
    ("rms_norm_quantize", _I, [_I, _P, _P, _P, _I, _I64, _I64, ctypes.c_double, _P, _P, _P, _P, _I, _P, _P]),
    ("rms_norm_vjp", _I, [_P, _P, _P, _P, _P, _I, _I64, _I64, _P, _P, _P, _SZ, _P]),
    ("rms_norm_vjp_workspace_size", _SZ, [_I64, _I64]),
    ("kv_cache_append", _I, [ctypes.POINTER(KvCacheArgs), _P, _P, _P, _I, _I64, _I64, _I64, _I64, _I64, _P, _P, _I64, _I64, _I,
                             _P, _P, _P, _P]),
    ("kv_cache_move", _I, [ctypes.POINTER(KvCacheArgs), _P, _P, _I64, _P, _I64, _P]),
    ("kv_attention_tree", _I, [ctypes.POINTER(KvCacheArgs), _P, _I, _I64, _P, _P, _P, _P, _I64, _I64, _I64, _I64, _I64, _I64,
                               _I64, ctypes.c_float, _I64, _P, _P, _P, _SZ, _P]),
    ("kv_cache_write", _I, [ctypes.POINTER(KvCacheArgs), _P, _P, _I, _I64, _I64, _I64, _P, _P]),
    ("kv_cache_read", _I, [ctypes.POINTER(KvCacheArgs), _P, _I64, _P, _P, _I, _P]),
    ("kv_attention", _I, [ctypes.POINTER(KvCacheArgs), _P, _I, _I64, _P, _P, _P, _I64, _I64, _I64, _I64, _I64, _I64,
                          ctypes.c_float, _I, _I64, _P, _P, _P, _SZ, _P]),
    ("kv_attention_workspace_size", _SZ, [_I64] * 8),
    ("kv_attention_tree_workspace_size", _SZ, [_I64] * 8),
]

_lib = None


class Nvfp4Error(RuntimeError):
    def __init__(self, status: int, message: str):
        super().__init__(f"{message} (status {status})")
        self.status = status


def lib():
    """The loaded libnvfp4.so (ctypes.CDLL) with argument types set."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(
                f"{LIB_PATH} is not built; run `python -m mxfp8_block_scaled_nvfp4_b200.build`")
        L = ctypes.CDLL(LIB_PATH)
        for name, res, args in SIGNATURES:
            f = getattr(L, name)
            f.restype = res
            f.argtypes = args
        _lib = L
    return _lib


def _check(status: int):
    if status != OK:
        L = lib()
        msg = L.nvfp4_last_error_message().decode() or L.nvfp4_status_string(status).decode()
        raise Nvfp4Error(status, msg)


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


# The raw handle of a device's current stream; building a torch.cuda.Stream
# object takes longer than a small launch.  (Not a public name of torch.)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda device: torch.cuda.current_stream(device).cuda_stream)


def _stream():
    """The current stream of the current device as a pointer."""
    return ctypes.c_void_p(_raw_stream(torch.cuda.current_device()))


def _need_cuda(*ts):
    """Every tensor is a contiguous CUDA tensor on the current device: the
    library launches on the current device and the current stream, so a
    tensor of another GPU would be read through a pointer that GPU's kernels
    cannot use.  Returns that device (None without a tensor)."""
    dev = None
    for t in ts:
        if t is not None:
            if not t.is_cuda:
                raise ValueError("tensors must be CUDA tensors (no CPU fallback)")
            if not t.is_contiguous():
                raise ValueError("tensors must be contiguous")
            if dev is None:
                dev = torch.cuda.current_device()
            if t.device.index != dev:
                raise ValueError(f"tensor on {t.device}, but the current device is cuda:{dev}; "
                                 "call under torch.cuda.device(tensor.device)")
    return dev


def _nbytes(t) -> int:
    return t.numel() * t.element_size()


def _need_bytes(t, nbytes: int, what: str):
    """The library takes raw pointers and cannot see a buffer's size: refuse
    one smaller than the bytes the call reads or writes through it."""
    if t is not None and _nbytes(t) < nbytes:
        raise ValueError(f"{what} holds {_nbytes(t)} bytes; the call needs {nbytes}")


def _need_dtype(t, dtype, what: str):
    if t is not None and t.dtype != dtype:
        raise ValueError(f"{what} must be {dtype}, got {t.dtype}")


def _need_g(g, n: int = 1, what: str = "global scale"):
    """Global scales are fp32 device scalars (n of them for per-expert g)."""
    _need_dtype(g, torch.float32, what)
    _need_bytes(g, 4 * n, what)


def _scale_nbytes(rows: int, cols: int, layout: str) -> int:
    r, c = scale_shape(rows, cols, layout)
    return r * c


def check_device_errors():
    _check(lib().nvfp4_check_device_errors(_stream()))


def scale_bytes(rows: int, cols: int, layout: str) -> int:
    return int(lib().nvfp4_scale_bytes(rows, cols, LAYOUT[layout]))


def scale_shape(rows: int, cols: int, layout: str):
    if layout == "linear":
        return (rows, cols)
    return ((rows + 127) // 128 * 128, (cols + 3) // 4 * 4)


# ---------------------------------------------------------------------------
def amax(x: torch.Tensor, out: torch.Tensor | None = None) -> torch.Tensor:
    """fp32 [1] tensor holding max |x| (the global scale g)."""
    _need_g(out, 1, "out")
    _need_cuda(x, out)
    out = torch.empty(1, dtype=torch.float32, device=x.device) if out is None else out
    _check(lib().nvfp4_amax(_ptr(x), DT[x.dtype], x.numel(), _ptr(out), _stream()))
    return out


def nvfp4_quantize(x: torch.Tensor, g: torch.Tensor | None = None, layout: str = "linear",
                   codes: torch.Tensor | None = None, scales: torch.Tensor | None = None):
    """(codes uint32 [rows, K/8] viewed as int32, scales uint8) of a 2-D x."""
    rows, K = x.shape
    _need_g(g)
    _need_bytes(codes, rows * (K // 8) * 4, "codes")
    _need_bytes(scales, _scale_nbytes(rows, K // 16, layout), "scales")
    _need_cuda(x, g, codes, scales)
    if codes is None:
        codes = torch.empty(rows, K // 8, dtype=torch.int32, device=x.device)
    if scales is None:
        scales = torch.empty(scale_shape(rows, K // 16, layout), dtype=torch.uint8, device=x.device)
    _check(lib().nvfp4_quantize(_ptr(x), DT[x.dtype], rows, K, _ptr(g), _ptr(codes), _ptr(scales),
                                LAYOUT[layout], _stream()))
    return codes, scales


def amax_multi(xs, out: torch.Tensor | None = None) -> torch.Tensor:
    """fp32 [len(xs)] tensor: out[i] = max |xs[i]|, one launch (1 to 4
    tensors of one dtype)."""
    n = len(xs)
    if not 1 <= n <= 4:
        raise ValueError("amax_multi takes 1 to 4 tensors")
    if any(x.dtype != xs[0].dtype for x in xs):
        raise ValueError("amax_multi: every tensor must have the same dtype")
    _need_g(out, n, "out")
    _need_cuda(*xs, out)
    out = torch.empty(n, dtype=torch.float32, device=xs[0].device) if out is None else out
    items = (AmaxItem * n)(*[AmaxItem(x.data_ptr(), x.numel(), out.data_ptr() + 4 * i) for i, x in enumerate(xs)])
    _check(lib().nvfp4_amax_multi(items, n, DT[xs[0].dtype], _stream()))
    return out


def nvfp4_quantize_multi(jobs):
    """nvfp4_quantize of 1 to 4 tensors of one dtype in one launch.  jobs:
    (x, g, layout[, codes, scales]) tuples, as nvfp4_quantize's arguments.
    Returns [(codes, scales), ...] in the same order."""
    n = len(jobs)
    if not 1 <= n <= 4:
        raise ValueError("nvfp4_quantize_multi takes 1 to 4 tensors")
    outs, items = [], []
    for job in jobs:
        x, g, layout = job[0], job[1], job[2]
        codes, scales = (job[3], job[4]) if len(job) > 3 else (None, None)
        if x.dtype != jobs[0][0].dtype:
            raise ValueError("nvfp4_quantize_multi: every tensor must have the same dtype")
        rows, K = x.shape
        _need_g(g)
        _need_bytes(codes, rows * (K // 8) * 4, "codes")
        _need_bytes(scales, _scale_nbytes(rows, K // 16, layout), "scales")
        _need_cuda(x, g, codes, scales)
        if codes is None:
            codes = torch.empty(rows, K // 8, dtype=torch.int32, device=x.device)
        if scales is None:
            scales = torch.empty(scale_shape(rows, K // 16, layout), dtype=torch.uint8, device=x.device)
        outs.append((codes, scales))
        items.append(QuantizeItem(x.data_ptr(), rows, K, None if g is None else g.data_ptr(), codes.data_ptr(),
                                  scales.data_ptr(), LAYOUT[layout]))
    arr = (QuantizeItem * n)(*items)
    _check(lib().nvfp4_quantize_multi(arr, n, DT[jobs[0][0].dtype], _stream()))
    return outs


def nvfp4_quantize_columnwise(x: torch.Tensor, g: torch.Tensor | None = None, layout: str = "linear",
                              codes: torch.Tensor | None = None, scales: torch.Tensor | None = None,
                              seed: int | None = None):
    """(codes [cols, rows/8], scales) of x^T quantized along the rows of a 2-D x
    (equal to nvfp4_quantize(x.T.contiguous(), g, layout)); with a seed,
    nvfp4_quantize_columnwise_sr (equal to nvfp4_quantize_sr of x^T)."""
    rows, cols = x.shape
    _need_g(g)
    _need_bytes(codes, cols * (rows // 8) * 4, "codes")
    _need_bytes(scales, _scale_nbytes(cols, rows // 16, layout), "scales")
    _need_cuda(x, g, codes, scales)
    if codes is None:
        codes = torch.empty(cols, rows // 8, dtype=torch.int32, device=x.device)
    if scales is None:
        scales = torch.empty(scale_shape(cols, rows // 16, layout), dtype=torch.uint8, device=x.device)
    if seed is None:
        _check(lib().nvfp4_quantize_columnwise(_ptr(x), DT[x.dtype], rows, cols, _ptr(g), _ptr(codes), _ptr(scales),
                                               LAYOUT[layout], _stream()))
    else:
        _check(lib().nvfp4_quantize_columnwise_sr(_ptr(x), DT[x.dtype], rows, cols, _ptr(g), seed, _ptr(codes),
                                                  _ptr(scales), LAYOUT[layout], _stream()))
    return codes, scales


def nvfp4_dequantize(codes: torch.Tensor, scales: torch.Tensor, g: torch.Tensor | None = None,
                     layout: str = "linear", dtype=torch.bfloat16, out: torch.Tensor | None = None) -> torch.Tensor:
    rows, K = codes.shape[0], codes.shape[1] * 8
    _need_g(g)
    _need_bytes(scales, _scale_nbytes(rows, K // 16, layout), "scales")
    _need_bytes(out, rows * K * (out.element_size() if out is not None else 0), "out")
    _need_cuda(codes, scales, g, out)
    if out is None:
        out = torch.empty(rows, K, dtype=dtype, device=codes.device)
    dtype = out.dtype
    _check(lib().nvfp4_dequantize(_ptr(codes), _ptr(scales), LAYOUT[layout], rows, K, _ptr(g), _ptr(out),
                                  DT[dtype], _stream()))
    return out


def nvfp4_quantize_sr(x: torch.Tensor, g: torch.Tensor | None = None, seed: int = 0, layout: str = "linear",
                      codes: torch.Tensor | None = None, scales: torch.Tensor | None = None):
    """nvfp4_quantize with stochastic rounding of the codes (Philox4x32-10
    random bits keyed by ``seed``); scales as nvfp4_quantize."""
    rows, K = x.shape
    _need_g(g)
    _need_bytes(codes, rows * (K // 8) * 4, "codes")
    _need_bytes(scales, _scale_nbytes(rows, K // 16, layout), "scales")
    _need_cuda(x, g, codes, scales)
    if codes is None:
        codes = torch.empty(rows, K // 8, dtype=torch.int32, device=x.device)
    if scales is None:
        scales = torch.empty(scale_shape(rows, K // 16, layout), dtype=torch.uint8, device=x.device)
    _check(lib().nvfp4_quantize_sr(_ptr(x), DT[x.dtype], rows, K, _ptr(g), seed, _ptr(codes), _ptr(scales),
                                   LAYOUT[layout], _stream()))
    return codes, scales


def mxfp8_quantize(x: torch.Tensor, layout: str = "linear", codes=None, scales=None):
    rows, K = x.shape
    _need_bytes(codes, rows * (K // 4) * 4, "codes")
    _need_bytes(scales, _scale_nbytes(rows, K // 32, layout), "scales")
    _need_cuda(x, codes, scales)
    if codes is None:
        codes = torch.empty(rows, K // 4, dtype=torch.int32, device=x.device)
    if scales is None:
        scales = torch.empty(scale_shape(rows, K // 32, layout), dtype=torch.uint8, device=x.device)
    _check(lib().mxfp8_quantize(_ptr(x), DT[x.dtype], rows, K, _ptr(codes), _ptr(scales), LAYOUT[layout],
                                _stream()))
    return codes, scales


def mxfp4_quantize(x: torch.Tensor, layout: str = "linear", codes=None, scales=None):
    """(codes int32 [rows, K/8], e8m0 scales uint8) of a 2-D x, 32-element blocks."""
    rows, K = x.shape
    _need_bytes(codes, rows * (K // 8) * 4, "codes")
    _need_bytes(scales, _scale_nbytes(rows, K // 32, layout), "scales")
    _need_cuda(x, codes, scales)
    if codes is None:
        codes = torch.empty(rows, K // 8, dtype=torch.int32, device=x.device)
    if scales is None:
        scales = torch.empty(scale_shape(rows, K // 32, layout), dtype=torch.uint8, device=x.device)
    _check(lib().mxfp4_quantize(_ptr(x), DT[x.dtype], rows, K, _ptr(codes), _ptr(scales), LAYOUT[layout],
                                _stream()))
    return codes, scales


def mxfp4_dequantize(codes, scales, layout: str = "linear", dtype=torch.bfloat16) -> torch.Tensor:
    rows, K = codes.shape[0], codes.shape[1] * 8
    _need_bytes(scales, _scale_nbytes(rows, K // 32, layout), "scales")
    _need_cuda(codes, scales)
    out = torch.empty(rows, K, dtype=dtype, device=codes.device)
    _check(lib().mxfp4_dequantize(_ptr(codes), _ptr(scales), LAYOUT[layout], rows, K, _ptr(out), DT[dtype],
                                  _stream()))
    return out


def mxfp8_dequantize(codes, scales, layout: str = "linear", dtype=torch.bfloat16) -> torch.Tensor:
    rows, K = codes.shape[0], codes.shape[1] * 4
    _need_bytes(scales, _scale_nbytes(rows, K // 32, layout), "scales")
    _need_cuda(codes, scales)
    out = torch.empty(rows, K, dtype=dtype, device=codes.device)
    _check(lib().mxfp8_dequantize(_ptr(codes), _ptr(scales), LAYOUT[layout], rows, K, _ptr(out), DT[dtype],
                                  _stream()))
    return out


def swizzle_scales(lin: torch.Tensor) -> torch.Tensor:
    _need_cuda(lin)
    rows, cols = lin.shape
    out = torch.empty(scale_shape(rows, cols, "swizzled"), dtype=torch.uint8, device=lin.device)
    _check(lib().nvfp4_swizzle_scales(_ptr(lin), rows, cols, _ptr(out), _stream()))
    return out


def qqmm(a_codes, a_scales, b_codes, b_scales, K: int, mode: str = "nvfp4", g_x=None, g_w=None,
         out_dtype=torch.bfloat16, out: torch.Tensor | None = None) -> torch.Tensor:
    """y [M, N] = x_hat . w_hat^T from quantized operands with SWIZZLED scales."""
    M, N = a_codes.shape[0], b_codes.shape[0]
    if mode in MODE:
        row_bytes = K if mode == "mxfp8" else K // 2
        group = 16 if mode == "nvfp4" else 32
        _need_bytes(a_codes, M * row_bytes, "a_codes")
        _need_bytes(b_codes, N * row_bytes, "b_codes")
        _need_bytes(a_scales, _scale_nbytes(M, K // group, "swizzled"), "a_scales")
        _need_bytes(b_scales, _scale_nbytes(N, K // group, "swizzled"), "b_scales")
    _need_g(g_x, 1, "g_x")
    _need_g(g_w, 1, "g_w")
    _need_bytes(out, M * N * (out.element_size() if out is not None else 0), "out")
    _need_cuda(a_codes, a_scales, b_codes, b_scales, g_x, g_w, out)
    if out is None:
        out = torch.empty(M, N, dtype=out_dtype, device=a_codes.device)
    _check(lib().qqmm(MODE[mode], M, N, K, _ptr(a_codes), _ptr(a_scales), _ptr(b_codes), _ptr(b_scales),
                      _ptr(g_x), _ptr(g_w), _ptr(out), DT[out.dtype], _stream()))
    return out


def qqmm_raw(x: torch.Tensor, w: torch.Tensor, out_dtype=None, out: torch.Tensor | None = None, buffers=None):
    """y [M, N] = qqmm of raw operands x [M, K] and w [N, K] (one dtype),
    NVFP4 with g = amax of each ("mlx 0.30.7.2 -> 0.30.7.6" diff, page 8,
    ops.cpp qqmm on unquantized inputs): both amaxes in one launch, both
    quantizations (SWIZZLED scales) in one launch, then the GEMM.  y has x's
    dtype unless out_dtype or out says otherwise.  buffers: optional
    preallocated (g [2] fp32, x codes, x scales, w codes, w scales)."""
    M, K = x.shape
    N = w.shape[0]
    if w.shape[1] != K or w.dtype != x.dtype:
        raise ValueError("x [M, K] and w [N, K] must share K and dtype")
    if buffers is None:
        dev = x.device
        g = torch.empty(2, dtype=torch.float32, device=dev)
        xc, wc = (torch.empty(r, K // 8, dtype=torch.int32, device=dev) for r in (M, N))
        xs, ws = (torch.empty(scale_shape(r, K // 16, "swizzled"), dtype=torch.uint8, device=dev) for r in (M, N))
    else:
        g, xc, xs, wc, ws = buffers
    amax_multi([x, w], g)
    nvfp4_quantize_multi([(x, g[0:1], "swizzled", xc, xs), (w, g[1:2], "swizzled", wc, ws)])
    return qqmm(xc, xs, wc, ws, K, "nvfp4", g[0:1], g[1:2], out_dtype=out_dtype or x.dtype, out=out)


def qqmm_vjp(x: torch.Tensor, w: torch.Tensor, cotan: torch.Tensor, g_x: torch.Tensor, g_w: torch.Tensor):
    """(dx, dw) of y = qqmm(x, w) ("mlx 0.30.7.2 -> 0.30.7.6" diff, page 8,
    QQMatmul::vjp, NVFP4 with global scales): with g_c = amax(cotan),
      dx = qqmm(cotan, w^T)   -- cotan quantized along N with g_c, w^T along N with g_w
      dw = qqmm(cotan^T, x^T) -- both quantized along M, with g_c and g_x.
    x [M, K], w [N, K], cotan [M, N] bf16/fp16/fp32; M, N multiples of 32.
    Every step is one ABI call (amax, quantize, column-wise quantize, qqmm)."""
    _need_cuda(x, w, cotan, g_x, g_w)
    M, N = x.shape[0], w.shape[0]
    g_c = amax(cotan)
    c_codes, c_scales = nvfp4_quantize(cotan, g_c, "swizzled")                # [M, N/8]
    wt_codes, wt_scales = nvfp4_quantize_columnwise(w, g_w, "swizzled")      # w^T [K, N/8]
    dx = qqmm(c_codes, c_scales, wt_codes, wt_scales, N, "nvfp4", g_c, g_w, out_dtype=x.dtype)
    ct_codes, ct_scales = nvfp4_quantize_columnwise(cotan, g_c, "swizzled")  # cotan^T [N, M/8]
    xt_codes, xt_scales = nvfp4_quantize_columnwise(x, g_x, "swizzled")      # x^T [K, M/8]
    dw = qqmm(ct_codes, ct_scales, xt_codes, xt_scales, M, "nvfp4", g_c, g_x, out_dtype=w.dtype)
    return dx, dw


def qmv(x: torch.Tensor, w_codes, w_scales, g_x=None, g_w=None, out=None, pdl: bool = False) -> torch.Tensor:
    """y [M, N] (x's dtype) = x_hat . w_hat^T, M <= 8, w pre-quantized (LINEAR scales).
    pdl=True calls qmv_pdl: for chains of decode calls whose weight (codes,
    scales, g_w) is not written by work still pending on the device."""
    M, K = x.shape
    N = w_codes.shape[0]
    _need_bytes(w_codes, N * (K // 8) * 4, "w_codes")
    _need_bytes(w_scales, N * (K // 16), "w_scales")
    _need_g(g_x, 1, "g_x")
    _need_g(g_w, 1, "g_w")
    _need_dtype(out, x.dtype, "out")
    _need_bytes(out, M * N * x.element_size(), "out")
    _need_cuda(x, w_codes, w_scales, g_x, g_w, out)
    if out is None:
        out = torch.empty(M, N, dtype=x.dtype, device=x.device)
    fn = lib().qmv_pdl if pdl else lib().qmv
    _check(fn(_ptr(x), DT[x.dtype], _ptr(g_x), _ptr(w_codes), _ptr(w_scales), _ptr(g_w), M, N, K, _ptr(out),
              _stream()))
    return out


def qmv_mx(x: torch.Tensor, w_codes, w_scales, mode: str, out=None) -> torch.Tensor:
    """y [M, N] (x's dtype) = x_hat . w_hat^T in an MX mode ("mxfp8": codes
    [N, K/4], "mxfp4": codes [N, K/8]; e8m0 scales LINEAR [N, K/32]), M <= 8."""
    if mode not in ("mxfp8", "mxfp4"):
        raise ValueError("qmv_mx: mode must be mxfp8 or mxfp4")
    M, K = x.shape
    N = w_codes.shape[0]
    _need_bytes(w_codes, N * (K if mode == "mxfp8" else K // 2), "w_codes")
    _need_bytes(w_scales, N * (K // 32), "w_scales")
    _need_dtype(out, x.dtype, "out")
    _need_bytes(out, M * N * x.element_size(), "out")
    _need_cuda(x, w_codes, w_scales, out)
    if out is None:
        out = torch.empty(M, N, dtype=x.dtype, device=x.device)
    _check(lib().qmv_mx(MODE[mode], _ptr(x), DT[x.dtype], _ptr(w_codes), _ptr(w_scales), M, N, K, _ptr(out),
                        _stream()))
    return out


def gather_qmm_workspace_size(T: int, topk: int, E: int) -> int:
    return int(lib().gather_qmm_workspace_size(T, topk, E))


def gather_qmm_staged_workspace_size(T: int, topk: int, E: int, K: int) -> int:
    return int(lib().gather_qmm_staged_workspace_size(T, topk, E, K))


def _need_gather(x, w_codes, w_scales, g, idx, out, T, topk, E, N, K, transpose):
    """Types and sizes the gather entries read and write through raw pointers."""
    _need_dtype(x, torch.bfloat16, "x")
    _need_dtype(idx, torch.int32, "idx")
    _need_bytes(idx, T * topk * 4, "idx")
    if transpose:
        _need_bytes(w_codes, E * N * (K // 8) * 4, "w_codes")
        _need_bytes(w_scales, E * N * (K // 16), "w_scales")
    else:
        _need_bytes(w_codes, E * K * (N // 8) * 4, "w_codes")
        _need_bytes(w_scales, E * K * (N // 16), "w_scales")
    _need_g(g, E, "g")
    _need_dtype(out, torch.bfloat16, "out")
    _need_bytes(out, T * topk * N * 2, "out")


def gather_qmm(x, w_codes, w_scales, g, idx, workspace=None, out=None, transpose: bool = True) -> torch.Tensor:
    """y [T, topk, N] bf16.  transpose=True: w_codes [E, N, K/8], w_scales
    LINEAR [E, N, K/16] (y = x . w_hat^T); transpose=False: w_codes
    [E, K, N/8], w_scales LINEAR [E, K, N/16] (y = x . w_hat)."""
    T, K = x.shape
    topk = idx.shape[1]
    E = w_codes.shape[0]
    N = w_codes.shape[1] if transpose else w_codes.shape[2] * 8
    _need_gather(x, w_codes, w_scales, g, idx, out, T, topk, E, N, K, transpose)
    _need_cuda(x, w_codes, w_scales, g, idx, workspace, out)
    if workspace is None:  # the staged form where it applies (weights [E, N, K])
        size = gather_qmm_staged_workspace_size(T, topk, E, K) if transpose else gather_qmm_workspace_size(T, topk, E)
        workspace = torch.empty(size, dtype=torch.uint8, device=x.device)
    if out is None:
        out = torch.empty(T, topk, N, dtype=torch.bfloat16, device=x.device)
    fn = lib().gather_qmm if transpose else lib().gather_qmm_kn
    _check(fn(_ptr(x), _ptr(w_codes), _ptr(w_scales), _ptr(g), _ptr(idx), T, topk, E, N, K,
              _ptr(out), _ptr(workspace), _nbytes(workspace), _stream()))
    return out


def gather_qmm_noalloc(x, w_codes, w_scales, g, idx, out=None) -> torch.Tensor:
    """gather_qmm using the library's own static scratch instead of a
    workspace (for callers that cannot allocate device memory); see
    include/nvfp4.h for its size limit and the rule that overlapping calls
    must be serialized."""
    T, K = x.shape
    topk = idx.shape[1]
    E, N = w_codes.shape[0], w_codes.shape[1]
    _need_gather(x, w_codes, w_scales, g, idx, out, T, topk, E, N, K, True)
    _need_cuda(x, w_codes, w_scales, g, idx, out)
    if out is None:
        out = torch.empty(T, topk, N, dtype=torch.bfloat16, device=x.device)
    _check(lib().gather_qmm_noalloc(_ptr(x), _ptr(w_codes), _ptr(w_scales), _ptr(g), _ptr(idx), T, topk, E, N, K,
                                    _ptr(out), _stream()))
    return out


# ---------------------------------------------------------------------------
# root-mean-square norm
# ---------------------------------------------------------------------------
def _need_norm(x, w, residual, h, rstd, *more):
    """Types and sizes of a norm's tensors; (rows, K, device) of x [..., K].
    (These calls are short: what is in order costs one comparison.)"""
    dtype = x.dtype
    if dtype not in DT:
        raise ValueError("x must be float32, float16 or bfloat16")
    if x.dim() < 1:
        raise ValueError("x must be [..., K]")
    K = x.shape[-1]
    rows = x.numel() // K if K else 0
    if w.dtype != dtype or w.numel() != K:
        _need_dtype(w, dtype, "weight")
        raise ValueError(f"weight must hold {K} elements, got {w.numel()}")
    if residual is not None:
        _need_like(residual, x, "residual")
        if h is not None:
            _need_like(h, x, "h")
    elif h is not None:
        raise ValueError("h is given with a residual, and only then")
    if rstd is not None:
        _need_dtype(rstd, torch.float32, "rstd")
        _need_bytes(rstd, 4 * rows, "rstd")
    return rows, K, _need_cuda(x, w, residual, h, rstd, *more)


def _need_like(t, x, what: str):
    _need_dtype(t, x.dtype, what)
    if t.shape != x.shape:
        raise ValueError(f"{what} must be {tuple(x.shape)}, got {tuple(t.shape)}")


def rms_norm(x: torch.Tensor, weight: torch.Tensor, eps: float = 1e-6, residual: torch.Tensor | None = None,
             out: torch.Tensor | None = None, h: torch.Tensor | None = None, rstd: torch.Tensor | None = None,
             return_rstd: bool = False):
    """(y, h): the norm's output y in x's dtype and what was normed, h = x +
    residual rounded to x's dtype (x itself without a residual), both of x's
    shape [..., K]; with return_rstd (or an rstd tensor) the triple (y, h,
    rstd), rstd fp32 [rows] for rms_norm_vjp.  h may be x or residual, to add
    in place."""
    if out is not None:
        _need_dtype(out, x.dtype, "out")
        _need_bytes(out, _nbytes(x), "out")
    rows, K, dev = _need_norm(x, weight, residual, h, rstd, out)
    if out is None:
        out = torch.empty_like(x)
    if residual is not None and h is None:
        h = torch.empty_like(x)
    if rstd is None and return_rstd:
        rstd = torch.empty(rows, dtype=torch.float32, device=x.device)
    _check(lib().rms_norm(x.data_ptr(), None if residual is None else residual.data_ptr(), weight.data_ptr(), DT[x.dtype], rows, K,
                          eps, None if h is None else h.data_ptr(), out.data_ptr(), None if rstd is None else rstd.data_ptr(),
                          _raw_stream(dev)))
    y = (out, x if h is None else h)
    return y if rstd is None else y + (rstd,)


def rms_norm_quantize(x: torch.Tensor, weight: torch.Tensor, mode: str, g: torch.Tensor | None = None, eps: float = 1e-6,
                      residual: torch.Tensor | None = None, layout: str = "linear", codes: torch.Tensor | None = None,
                      scales: torch.Tensor | None = None, h: torch.Tensor | None = None, rstd: torch.Tensor | None = None,
                      return_rstd: bool = False):
    """(codes, scales, h): rms_norm's fp32 output quantized as mode's quantizer
    does (codes int32 [rows, K/8], "mxfp8" K/4; scales uint8 in `layout`; g the
    fp32 [1] amax of the output, "nvfp4" only), and h as rms_norm gives it; with
    return_rstd (or an rstd tensor) rstd as well."""
    if mode not in MODE:
        raise ValueError("rms_norm_quantize: mode must be nvfp4, mxfp8 or mxfp4")
    if g is not None:
        _need_g(g, 1, "g")
    rows, K, dev = _need_norm(x, weight, residual, h, rstd, g, codes, scales)
    per, group = 4 if mode == "mxfp8" else 8, 16 if mode == "nvfp4" else 32
    if codes is None:
        codes = torch.empty(rows, K // per, dtype=torch.int32, device=x.device)
    else:
        _need_bytes(codes, rows * (K // per) * 4, "codes")
    shape = scale_shape(rows, K // group, layout)
    if scales is None:
        scales = torch.empty(shape, dtype=torch.uint8, device=x.device)
    else:
        _need_bytes(scales, shape[0] * shape[1], "scales")
    if residual is not None and h is None:
        h = torch.empty_like(x)
    if rstd is None and return_rstd:
        rstd = torch.empty(rows, dtype=torch.float32, device=x.device)
    _check(lib().rms_norm_quantize(
        MODE[mode], x.data_ptr(), None if residual is None else residual.data_ptr(), weight.data_ptr(), DT[x.dtype], rows, K, eps,
        None if g is None else g.data_ptr(), None if h is None else h.data_ptr(), codes.data_ptr(), scales.data_ptr(),
        LAYOUT[layout], None if rstd is None else rstd.data_ptr(), _raw_stream(dev)))
    y = (codes, scales, x if h is None else h)
    return y if rstd is None else y + (rstd,)


@functools.lru_cache(maxsize=4096)
def rms_norm_vjp_workspace_size(rows: int, K: int) -> int:
    return int(lib().rms_norm_vjp_workspace_size(rows, K))


def rms_norm_vjp(dy: torch.Tensor, h: torch.Tensor, weight: torch.Tensor, rstd: torch.Tensor,
                 dh: torch.Tensor | None = None, dx: torch.Tensor | None = None, dw: torch.Tensor | None = None,
                 workspace: torch.Tensor | None = None):
    """(dx, dw): gradients of rms_norm and rms_norm_quantize (which passes the
    gradient of its output straight through).  dy: gradient of the output; h,
    rstd as the forward call gave them; dh: gradient that reaches h past the
    norm (None: none).  dx (dy's dtype; it may be dy or dh) is the gradient of
    x and of residual; dw fp32 [K] that of weight."""
    _need_like(h, dy, "h")
    if dx is not None:
        _need_dtype(dx, dy.dtype, "dx")
        _need_bytes(dx, _nbytes(dy), "dx")
    rows, K, dev = _need_norm(dy, weight, dh, None, rstd, h, dx, dw, workspace)
    if dw is not None:
        _need_dtype(dw, torch.float32, "dw")
        _need_bytes(dw, 4 * K, "dw")
    if dx is None:
        dx = torch.empty_like(dy)
    if dw is None:
        dw = torch.empty(K, dtype=torch.float32, device=dy.device)
    if workspace is None:
        workspace = torch.empty(rms_norm_vjp_workspace_size(rows, K), dtype=torch.uint8, device=dy.device)
    _check(lib().rms_norm_vjp(dy.data_ptr(), h.data_ptr(), weight.data_ptr(), rstd.data_ptr(), None if dh is None else dh.data_ptr(),
                              DT[dy.dtype], rows, K, dx.data_ptr(), dw.data_ptr(), workspace.data_ptr(), workspace.nbytes,
                              _raw_stream(dev)))
    return dx, dw


# ---------------------------------------------------------------------------
# key/value cache
# ---------------------------------------------------------------------------
class KvCache:
    """Handle of a paged key/value cache (nvfp4_kv_cache): the caller's tensors
    and the sizes they hold.  codes int32 [num_pages, heads, page_size, D/8]
    (D/4 for "mxfp8"), scales uint8 [num_pages, heads, page_size, D/16]
    ("nvfp4") or D/32; g_k, g_v fp32 [1] or None ("nvfp4" only, both or
    neither).  The handle keeps references to the tensors and no copy, and
    their addresses with them: its attributes cannot be set (a cache in other
    tensors is another handle), and the tensors' storage must stay in place."""

    def __init__(self, mode: str, k_codes, k_scales, v_codes, v_scales, g_k=None, g_v=None):
        if mode not in MODE:
            raise ValueError("KvCache: mode must be nvfp4, mxfp8 or mxfp4")
        if k_codes.dim() != 4:
            raise ValueError("KvCache: codes must be [num_pages, heads, page_size, words]")
        P, H, R, words = k_codes.shape
        D = words * (4 if mode == "mxfp8" else 8)
        sshape = (P, H, R, D // (16 if mode == "nvfp4" else 32))
        for t, what, dtype, shape in ((k_codes, "k_codes", torch.int32, k_codes.shape),
                                      (v_codes, "v_codes", torch.int32, k_codes.shape),
                                      (k_scales, "k_scales", torch.uint8, sshape),
                                      (v_scales, "v_scales", torch.uint8, sshape)):
            _need_dtype(t, dtype, what)
            if tuple(t.shape) != tuple(shape):
                raise ValueError(f"{what} must be {tuple(shape)}, got {tuple(t.shape)}")
        _need_g(g_k, 1, "g_k")
        _need_g(g_v, 1, "g_v")
        _need_cuda(k_codes, k_scales, v_codes, v_scales, g_k, g_v)
        args = KvCacheArgs(MODE[mode], P, R, H, D, *(None if t is None else t.data_ptr() for t in (
            k_codes, k_scales, v_codes, v_scales, g_k, g_v)))
        self.__dict__.update(mode=mode, num_pages=P, heads=H, page_size=R, D=D, k_codes=k_codes, k_scales=k_scales,
                             v_codes=v_codes, v_scales=v_scales, g_k=g_k, g_v=g_v, device=k_codes.device, _index=k_codes.device.index, _args=args,
                             _ref=ctypes.byref(args))

    def __setattr__(self, name, value):
        raise AttributeError(f"KvCache.{name} cannot be set: the handle holds its tensors' addresses; make a new one")

    def __delattr__(self, name):
        raise AttributeError(f"KvCache.{name} cannot be deleted")

    @classmethod
    def empty(cls, mode: str, num_pages: int, heads: int, page_size: int, D: int, g_k=None, g_v=None, device="cuda"):
        """A cache in new tensors (contents undefined until written)."""
        if mode not in MODE:
            raise ValueError("KvCache: mode must be nvfp4, mxfp8 or mxfp4")
        t = []
        for _ in range(2):
            t.append(torch.empty(num_pages, heads, page_size, D // (4 if mode == "mxfp8" else 8), dtype=torch.int32,
                                 device=device))
            t.append(torch.empty(num_pages, heads, page_size, D // (16 if mode == "nvfp4" else 32), dtype=torch.uint8,
                                 device=device))
        return cls(mode, *t, g_k, g_v)


def _need_rows(t, shape, what: str, dev: int):
    """[T, heads, D] on the current device `dev`, heads and D contiguous, any
    token stride (a part of a longer row is taken as it is)."""
    if t.shape != shape:
        raise ValueError(f"{what} must be {shape}, got {tuple(t.shape)}")
    if not t.is_cuda:
        raise ValueError("tensors must be CUDA tensors (no CPU fallback)")
    if t.device.index != dev:
        raise ValueError(f"{what} on {t.device}, but the current device is cuda:{dev}; "
                         "call under torch.cuda.device(tensor.device)")
    st = t.stride()
    if t.numel() and ((st[2] != 1 and shape[2] > 1) or (st[1] != shape[2] and shape[1] > 1)):
        raise ValueError(f"{what}: heads and D must be contiguous")
    return st[0]


def _need_cache(cache) -> int:
    """The current device, which has to be the cache's."""
    dev = torch.cuda.current_device()
    if cache._index != dev:
        raise ValueError(f"the cache is on {cache.device}, but the current device is cuda:{dev}; "
                         "call under torch.cuda.device(cache.device)")
    return dev


def kv_cache_write(cache: KvCache, k: torch.Tensor, v: torch.Tensor, slots: torch.Tensor) -> None:
    """Quantize k, v [T, heads, D] (one dtype; any token stride) into the
    cache's slots [T] int32 (negative: skipped)."""
    shape = (slots.shape[0], cache.heads, cache.D)
    if k.dtype != v.dtype or k.dtype not in DT:
        raise ValueError("k and v must share a dtype: float32, float16 or bfloat16")
    _need_dtype(slots, torch.int32, "slots")
    _need_cuda(slots)
    dev = _need_cache(cache)
    k_stride, v_stride = _need_rows(k, shape, "k", dev), _need_rows(v, shape, "v", dev)
    _check(lib().kv_cache_write(cache._ref, k.data_ptr(), v.data_ptr(), DT[k.dtype], shape[0], k_stride, v_stride,
                                slots.data_ptr(), _stream()))


def kv_cache_append(cache: KvCache, q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, cos: torch.Tensor,
                    sin: torch.Tensor, positions: torch.Tensor, slots: torch.Tensor, interleaved: bool = False,
                    q_out: torch.Tensor | None = None) -> torch.Tensor:
    """Rotate the queries q [T, Hq, D] and keys k [T, heads, D] of T new tokens
    by their positions [T] int32 and quantize keys and values into the cache's
    slots [T] int32; returns the rotated queries [T, Hq, D] (q's dtype,
    contiguous).  cos, sin fp32 [max_pos, rot / 2]: the first rot elements of a
    head turn, in pairs (i, i + rot / 2) or, interleaved, (2i, 2i + 1).  A token
    with a negative slot is skipped, its row of q_out left as it is."""
    T, heads, D = slots.shape[0], cache.heads, cache.D
    if q.dim() != 3:
        raise ValueError("q must be [T, Hq, D]")
    Hq = q.shape[1]
    dtype = q.dtype
    if dtype != k.dtype or dtype != v.dtype or dtype not in DT:
        raise ValueError("q, k and v must share a dtype: float32, float16 or bfloat16")
    _need_dtype(slots, torch.int32, "slots")
    _need_dtype(positions, torch.int32, "positions")
    _need_dtype(cos, torch.float32, "cos")
    _need_dtype(sin, torch.float32, "sin")
    if cos.dim() != 2 or cos.shape != sin.shape:
        raise ValueError("cos and sin must both be [max_pos, rot / 2]")
    if positions.numel() < T:
        _need_bytes(positions, 4 * T, "positions")
    if q_out is not None:
        _need_dtype(q_out, dtype, "q_out")
        _need_bytes(q_out, T * Hq * D * q.element_size(), "q_out")
    _need_cuda(slots, positions, cos, sin, q_out)
    dev, shape = _need_cache(cache), (T, heads, D)
    q_stride, k_stride, v_stride = _need_rows(q, (T, Hq, D), "q", dev), _need_rows(k, shape, "k", dev), _need_rows(v, shape, "v", dev)
    if q_out is None:
        q_out = torch.empty_like(q, memory_format=torch.contiguous_format)
    most, half = cos.shape
    _check(lib().kv_cache_append(cache._ref, q.data_ptr(), k.data_ptr(), v.data_ptr(), DT[dtype], T, Hq, q_stride, k_stride, v_stride,
                                 cos.data_ptr(), sin.data_ptr(), most, 2 * half, interleaved, positions.data_ptr(),
                                 slots.data_ptr(), q_out.data_ptr(), _raw_stream(dev)))
    return q_out


def kv_cache_move(cache: KvCache, src: torch.Tensor, dst: torch.Tensor, starts: torch.Tensor | None = None) -> None:
    """Copy the rows of slots src [M] to slots dst [M] (int32; a negative one
    skips its move).  starts [S + 1] int32: the moves starts[s] .. starts[s + 1]
    - 1 of a sequence take effect one after the other, as a chain; None: every
    move for itself (no slot is then both written and read or written twice),
    many times faster for long copies."""
    M = src.shape[0]
    _need_dtype(src, torch.int32, "src")
    _need_dtype(dst, torch.int32, "dst")
    _need_dtype(starts, torch.int32, "starts")
    if dst.shape != src.shape or src.dim() != 1:
        raise ValueError("src and dst must both be [M]")
    if starts is not None and (starts.dim() != 1 or starts.shape[0] < 1):
        raise ValueError("starts must be [S + 1]")
    _need_cuda(src, dst, starts)
    dev = _need_cache(cache)
    _check(lib().kv_cache_move(cache._ref, src.data_ptr(), dst.data_ptr(), M, None if starts is None else starts.data_ptr(),
                               M if starts is None else starts.shape[0] - 1, _raw_stream(dev)))


def kv_cache_read(cache: KvCache, slots: torch.Tensor, dtype=torch.bfloat16, k_out=None, v_out=None):
    """(k, v) [T, heads, D]: the values of the slots [T] int32 (negative: zero
    rows)."""
    shape = (slots.shape[0], cache.heads, cache.D)
    _need_dtype(slots, torch.int32, "slots")
    if k_out is None:
        k_out = torch.empty(shape, dtype=dtype, device=slots.device)
    if v_out is None:
        v_out = torch.empty_like(k_out)
    if k_out.dtype != v_out.dtype or k_out.dtype not in DT:
        raise ValueError("k_out and v_out must share a dtype: float32, float16 or bfloat16")
    for t, what in ((k_out, "k_out"), (v_out, "v_out")):
        if t.shape != shape:
            raise ValueError(f"{what} must be {shape}, got {tuple(t.shape)}")
    _need_cuda(slots, k_out, v_out)
    dev = _need_cache(cache)
    _check(lib().kv_cache_read(cache._ref, slots.data_ptr(), shape[0], k_out.data_ptr(), v_out.data_ptr(),
                               DT[k_out.dtype], _raw_stream(dev)))
    return k_out, v_out


@functools.lru_cache(maxsize=4096)
def kv_attention_workspace_size(B: int, T: int, Hq: int, heads: int, D: int, max_q: int = 1, max_kv: int = 0,
                                window: int = 0) -> int:
    return int(lib().kv_attention_workspace_size(B, T, Hq, heads, D, max_q, max_kv, window))


def kv_attention(cache: KvCache, q: torch.Tensor, page_table: torch.Tensor, kv_len: torch.Tensor,
                 q_start: torch.Tensor | None = None, max_q: int | None = None, max_kv: int | None = None,
                 scale: float | None = None, causal: bool = True, window: int = 0, out: torch.Tensor | None = None,
                 lse: torch.Tensor | None = None, return_lse: bool = False, workspace: torch.Tensor | None = None):
    """out [T, Hq, D] (q's dtype) = attention of the queries q [T, Hq, D] (fp16
    or bf16) over the cached tokens of their sequences; with return_lse (or an
    lse tensor [T, Hq] fp32) the pair (out, lse).
    page_table [B, max_pages] int32, kv_len [B] int32 (the queries' own tokens
    included).  q_start [B + 1] int32: sequence b has tokens q_start[b] ..
    q_start[b + 1] - 1 (None: one query a sequence).  max_q, max_kv: host
    bounds on queries and cached tokens of a sequence (default: T and all of
    the page table; tight bounds are faster).  scale defaults to D ** -0.5.
    workspace: uint8 scratch of kv_attention_workspace_size bytes (allocated
    here when None)."""
    T, Hq, D = q.shape
    B, max_pages = page_table.shape
    # (what is None is not looked at: a decoding call is short)
    if page_table.dtype != torch.int32 or kv_len.dtype != torch.int32 or kv_len.numel() < B:
        _need_dtype(page_table, torch.int32, "page_table")
        _need_dtype(kv_len, torch.int32, "kv_len")
        _need_bytes(kv_len, 4 * B, "kv_len")
    _need_cuda(page_table, kv_len)
    if q_start is not None:
        _need_dtype(q_start, torch.int32, "q_start")
        _need_bytes(q_start, 4 * (B + 1), "q_start")
        _need_cuda(q_start)
    if out is not None:
        _need_dtype(out, q.dtype, "out")
        _need_bytes(out, T * Hq * D * q.element_size(), "out")
        _need_cuda(out)
    if lse is not None:
        _need_dtype(lse, torch.float32, "lse")
        _need_bytes(lse, 4 * T * Hq, "lse")
        _need_cuda(lse)
    if workspace is not None:
        _need_cuda(workspace)
    q_stride = _need_rows(q, (T, Hq, cache.D), "q", _need_cache(cache))
    if q.dtype not in (torch.float16, torch.bfloat16):
        raise ValueError(f"q must be float16 or bfloat16, got {q.dtype}")
    if max_q is None:
        max_q = 1 if q_start is None else T
    if max_kv is None:
        max_kv = max_pages * cache.page_size
    if out is None:
        out = torch.empty_like(q, memory_format=torch.contiguous_format)
    if lse is None and return_lse:
        lse = torch.empty(T, Hq, dtype=torch.float32, device=q.device)
    if workspace is None:
        size = kv_attention_workspace_size(B, T, Hq, cache.heads, cache.D, max_q, max_kv, window)
        workspace = torch.empty(size, dtype=torch.uint8, device=cache.device) if size else None
    else:
        size = _nbytes(workspace)
    _check(lib().kv_attention(
        cache._ref, q.data_ptr(), DT[q.dtype], q_stride, None if q_start is None else q_start.data_ptr(),
        kv_len.data_ptr(), page_table.data_ptr(), B, T, Hq, max_q, max_kv, max_pages,
        cache.D ** -0.5 if scale is None else scale, causal, window, out.data_ptr(),
        None if lse is None else lse.data_ptr(), None if workspace is None else workspace.data_ptr(), size, _stream()))
    return out if lse is None else (out, lse)


@functools.lru_cache(maxsize=4096)
def kv_attention_tree_workspace_size(B: int, T: int, Hq: int, heads: int, D: int, max_q: int = 1, max_kv: int = 0,
                                     window: int = 0) -> int:
    return int(lib().kv_attention_tree_workspace_size(B, T, Hq, heads, D, max_q, max_kv, window))


def kv_attention_tree(cache: KvCache, q: torch.Tensor, page_table: torch.Tensor, kv_len: torch.Tensor,
                      tree_mask: torch.Tensor, q_start: torch.Tensor, max_q: int | None = None, max_kv: int | None = None,
                      scale: float | None = None, window: int = 0, out: torch.Tensor | None = None,
                      lse: torch.Tensor | None = None, return_lse: bool = False, workspace: torch.Tensor | None = None):
    """kv_attention for drafted tokens that form trees: the queries q
    [q_start[b] .. q_start[b + 1]) are the last of sequence b's kv_len[b] cached
    tokens, and each sees the context before them and of them those in its row
    of tree_mask [T, words] int32 (bit d % 32 of word d / 32: draft d, itself
    included only where its bit is set; 32 * words >= max_q, the host bound on a
    sequence's drafts and by default as many as the masks hold).  window: the
    context within window tokens of the query's place in its branch (the number
    of drafts it sees, less one).  workspace: uint8 scratch of
    kv_attention_tree_workspace_size bytes (allocated here when None).  The rest
    as in kv_attention."""
    T, Hq, D = q.shape
    B, max_pages = page_table.shape
    # (what is None is not looked at: a decoding call is short)
    if page_table.dtype != torch.int32 or kv_len.dtype != torch.int32 or kv_len.numel() < B:
        _need_dtype(page_table, torch.int32, "page_table")
        _need_dtype(kv_len, torch.int32, "kv_len")
        _need_bytes(kv_len, 4 * B, "kv_len")
    _need_dtype(q_start, torch.int32, "q_start")
    _need_bytes(q_start, 4 * (B + 1), "q_start")
    if tree_mask.dtype != torch.int32 and tree_mask.dtype != torch.uint32:
        raise ValueError(f"tree_mask must be {torch.int32}, got {tree_mask.dtype}")
    if tree_mask.dim() != 2 or tree_mask.shape[0] != T:
        raise ValueError(f"tree_mask must be [{T}, words], got {tuple(tree_mask.shape)}")
    _need_cuda(page_table, kv_len, q_start, tree_mask)
    if out is not None:
        _need_dtype(out, q.dtype, "out")
        _need_bytes(out, T * Hq * D * q.element_size(), "out")
        _need_cuda(out)
    if lse is not None:
        _need_dtype(lse, torch.float32, "lse")
        _need_bytes(lse, 4 * T * Hq, "lse")
        _need_cuda(lse)
    if workspace is not None:
        _need_cuda(workspace)
    q_stride = _need_rows(q, (T, Hq, cache.D), "q", _need_cache(cache))
    if q.dtype not in (torch.float16, torch.bfloat16):
        raise ValueError(f"q must be float16 or bfloat16, got {q.dtype}")
    if max_q is None:
        max_q = min(T, 32 * tree_mask.shape[1])
    if max_kv is None:
        max_kv = max_pages * cache.page_size
    if out is None:
        out = torch.empty_like(q, memory_format=torch.contiguous_format)
    if lse is None and return_lse:
        lse = torch.empty(T, Hq, dtype=torch.float32, device=q.device)
    if workspace is None:
        size = kv_attention_tree_workspace_size(B, T, Hq, cache.heads, cache.D, max_q, max_kv, window)
        workspace = torch.empty(size, dtype=torch.uint8, device=cache.device) if size else None
    else:
        size = _nbytes(workspace)
    _check(lib().kv_attention_tree(
        cache._ref, q.data_ptr(), DT[q.dtype], q_stride, q_start.data_ptr(), kv_len.data_ptr(), page_table.data_ptr(),
        tree_mask.data_ptr(), tree_mask.shape[1], B, T, Hq, max_q, max_kv, max_pages,
        cache.D ** -0.5 if scale is None else scale, window, out.data_ptr(),
        None if lse is None else lse.data_ptr(), None if workspace is None else workspace.data_ptr(), size, _stream()))
    return out if lse is None else (out, lse)
