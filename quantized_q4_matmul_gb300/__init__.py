"""Python binding of libqk, the GB300 (sm_103a) quantized Q4_K / Q6_K matmul library.

This module only marshals arguments: every step of the computation runs in the
CUDA kernels behind the C ABI declared in ``include/qk.h``.  Functions take
torch tensors (device memory) or raw integer addresses, plus an optional CUDA
stream (default: torch's current stream), and raise ``QKError`` on any non-zero
status.  A tensor argument must be contiguous and large enough for the call
(x and fp16 outputs fp16, or its bits as int16 / uint16; fp32 outputs
float32), else ``ValueError`` is raised before the library is called; raw
addresses are the caller's responsibility.  There is no CPU fallback: if ``libqk.so`` is missing or cannot be
loaded, every call raises.
"""
from __future__ import annotations

import ctypes
import os

__all__ = [
    "QKError", "lib", "lib_path", "qk_dequant_q4k", "qk_dequant_q6k", "qk_matmul_q4k", "qk_matmul_q6k",
    "qk_gateup_swiglu_q4k", "qk_matmul_batch", "qk_matmul_batch_q8x", "qk_matmul_q8x_q4k", "qk_matmul_q8x_q6k",
    "qk_get_device_status", "qk_debug_wait_timeout",
    "qk_decode_uses_gemv", "qk_uses_gemv", "qk_gemm_plan", "qk_rmsnorm_matmul_batch", "qk_rmsnorm_matmul_q4k",
    "qk_rmsnorm_matmul_q6k", "qk_rmsnorm_gateup_swiglu_q4k", "qk_rmsnorm_scratch_bytes",
    "qk_rmsnorm_matmul_batch_static", "qk_status_string", "qk_version", "QK_BLOCK_BYTES", "qk_matmul_desc",
    "qk_gemm_plan_info", "qk_gqa_attention", "qk_gqa_attention_window", "qk_matmul_batch_q8", "qk_matmul_q8_desc",
    "qk_add_rmsnorm", "qk_add_rmsnorm_q8", "qk_rope_kv_append", "qk_rope_inv_freq", "qk_rope_config", "qk_logprobs",
    "QK_F16", "QK_F32", "QK_ROPE_INTERLEAVED", "QK_ROPE_HALF", "QK_ROPE_SCALE_NONE", "QK_ROPE_SCALE_LINEAR",
    "QK_ROPE_SCALE_BANDED", "qk_norm_rope_kv_append", "qk_norm_rope_kv_append_q4", "qk_dequant_kv_q4",
    "qk_gqa_attention_q4", "qk_gqa_attention_q4_scratch_bytes", "qk_sample",
]

_HERE = os.path.dirname(os.path.abspath(__file__))
QK_BLOCK_BYTES = {"q4k": 144, "q6k": 210}

SYMBOLS = ("qk_dequant_q4k", "qk_dequant_q6k", "qk_matmul_q4k", "qk_matmul_q6k", "qk_gateup_swiglu_q4k",
           "qk_matmul_batch", "qk_matmul_batch_q8x", "qk_matmul_q8x_q4k", "qk_matmul_q8x_q6k",
           "qk_get_device_status", "qk_debug_wait_timeout", "qk_decode_uses_gemv",
           "qk_uses_gemv", "qk_gemm_plan", "qk_rmsnorm_matmul_batch", "qk_rmsnorm_matmul_q4k",
           "qk_rmsnorm_matmul_q6k", "qk_rmsnorm_gateup_swiglu_q4k", "qk_rmsnorm_scratch_bytes",
    "qk_rmsnorm_matmul_batch_static", "qk_status_string",
           "qk_version", "qk_gqa_attention", "qk_gqa_attention_window", "qk_matmul_batch_q8", "qk_add_rmsnorm",
           "qk_add_rmsnorm_q8", "qk_rope_kv_append", "qk_rope_inv_freq", "qk_logprobs", "qk_norm_rope_kv_append",
           "qk_norm_rope_kv_append_q4", "qk_dequant_kv_q4", "qk_gqa_attention_q4", "qk_gqa_attention_q4_scratch_bytes",
           "qk_sample")

QK_Q4_K, QK_Q6_K = 0, 1
_QTYPES = {"q4k": QK_Q4_K, "q6k": QK_Q6_K}
QK_F16, QK_F32 = 0, 1
QK_ROPE_INTERLEAVED, QK_ROPE_HALF = 0, 1
QK_ROPE_SCALE_NONE, QK_ROPE_SCALE_LINEAR, QK_ROPE_SCALE_BANDED = 0, 1, 2


class qk_matmul_desc(ctypes.Structure):
    """Mirror of ``qk_matmul_desc`` in include/qk.h."""
    _fields_ = [("qtype", ctypes.c_int), ("blocks", ctypes.c_void_p), ("up_blocks", ctypes.c_void_p),
                ("x_f16", ctypes.c_void_p), ("y", ctypes.c_void_p), ("M", ctypes.c_int64),
                ("N", ctypes.c_int64), ("K", ctypes.c_int64)]


class qk_matmul_q8_desc(ctypes.Structure):
    """Mirror of ``qk_matmul_q8_desc`` in include/qk.h."""
    _fields_ = [("qtype", ctypes.c_int), ("blocks", ctypes.c_void_p), ("up_blocks", ctypes.c_void_p),
                ("x_q8", ctypes.c_void_p), ("x_d", ctypes.c_void_p), ("y", ctypes.c_void_p), ("M", ctypes.c_int64),
                ("N", ctypes.c_int64), ("K", ctypes.c_int64)]


class qk_rope_config(ctypes.Structure):
    """Mirror of ``qk_rope_config`` in include/qk.h."""
    _fields_ = [("theta", ctypes.c_double), ("scaling", ctypes.c_int), ("factor", ctypes.c_double),
                ("low_turns", ctypes.c_double), ("high_turns", ctypes.c_double), ("original_len", ctypes.c_int64),
                ("freq_factors", ctypes.POINTER(ctypes.c_float))]


class qk_gemm_plan_info(ctypes.Structure):
    """Mirror of ``qk_gemm_plan_info`` in include/qk.h."""
    _fields_ = [(n, ctypes.c_int) for n in ("token_tile", "x_stages", "a_stages", "packed_stages", "a_in_tmem",
                                             "tmem_cols", "smem_bytes", "max_ctas_per_sm")]


class QKError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__("%s failed: %s (%d)" % (where, qk_status_string(status), status))


def lib_path() -> str:
    return os.environ.get("QK_LIB", os.path.join(_HERE, "libqk.so"))


_lib = None


def lib():
    """The loaded libqk (raises if it has not been built)."""
    global _lib
    if _lib is None:
        path = lib_path()
        if not os.path.exists(path):
            raise RuntimeError("libqk.so not found at %s: build it with "
                               "`python -c 'import __graft_entry__ as g; g.build()'`" % path)
        L = ctypes.CDLL(path)
        vp, i64, i32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int
        for name in ("qk_dequant_q4k", "qk_dequant_q6k"):
            f = getattr(L, name)
            f.restype, f.argtypes = i32, [vp, i64, vp, vp]
        for name in ("qk_matmul_q4k", "qk_matmul_q6k"):
            f = getattr(L, name)
            f.restype, f.argtypes = i32, [vp, vp, vp, i64, i64, i64, vp]
        L.qk_gateup_swiglu_q4k.restype = i32
        L.qk_gateup_swiglu_q4k.argtypes = [vp, vp, vp, vp, i64, i64, i64, vp]
        L.qk_matmul_batch.restype = i32
        L.qk_matmul_batch.argtypes = [ctypes.POINTER(qk_matmul_desc), i32, vp]
        L.qk_matmul_batch_q8x.restype = i32
        L.qk_matmul_batch_q8x.argtypes = [ctypes.POINTER(qk_matmul_desc), i32, vp]
        for f in (L.qk_matmul_q8x_q4k, L.qk_matmul_q8x_q6k):
            f.restype, f.argtypes = i32, [vp, vp, vp, i64, i64, i64, vp]
        L.qk_get_device_status.restype, L.qk_get_device_status.argtypes = i32, [vp]
        L.qk_debug_wait_timeout.restype, L.qk_debug_wait_timeout.argtypes = i32, [i64, vp]
        L.qk_decode_uses_gemv.restype, L.qk_decode_uses_gemv.argtypes = i32, [i32, i32, i64]
        L.qk_uses_gemv.restype, L.qk_uses_gemv.argtypes = i32, [i32, i32, i64, i64]
        f32 = ctypes.c_float
        L.qk_rmsnorm_matmul_batch.restype = i32
        L.qk_rmsnorm_matmul_batch.argtypes = [ctypes.POINTER(qk_matmul_desc), i32, vp, f32, vp, vp]
        for name in ("qk_rmsnorm_matmul_q4k", "qk_rmsnorm_matmul_q6k"):
            f = getattr(L, name)
            f.restype, f.argtypes = i32, [vp, vp, vp, f32, vp, vp, i64, i64, i64, vp]
        L.qk_rmsnorm_gateup_swiglu_q4k.restype = i32
        L.qk_rmsnorm_gateup_swiglu_q4k.argtypes = [vp, vp, vp, vp, f32, vp, vp, i64, i64, i64, vp]
        L.qk_rmsnorm_scratch_bytes.restype, L.qk_rmsnorm_scratch_bytes.argtypes = i64, [i32, i32, i64, i64]
        L.qk_rmsnorm_matmul_batch_static.restype = i32
        L.qk_rmsnorm_matmul_batch_static.argtypes = [ctypes.POINTER(qk_matmul_desc), i32, vp, f32, vp]
        L.qk_gemm_plan.restype = i32
        L.qk_gemm_plan.argtypes = [i32, i32, i64, i64, i64, ctypes.POINTER(qk_gemm_plan_info)]
        L.qk_gqa_attention.restype = i32
        L.qk_gqa_attention.argtypes = [vp, vp, vp, vp, i64, i64, i64, i64, i64, i64, f32, vp]
        L.qk_gqa_attention_window.restype = i32
        L.qk_gqa_attention_window.argtypes = [vp, vp, vp, vp, i64, i64, i64, i64, i64, i64, f32, i64, i64, vp]
        L.qk_matmul_batch_q8.restype = i32
        L.qk_matmul_batch_q8.argtypes = [ctypes.POINTER(qk_matmul_q8_desc), i32, vp]
        L.qk_add_rmsnorm.restype = i32
        L.qk_add_rmsnorm.argtypes = [vp, i32, vp, vp, f32, vp, vp, i64, i64, vp]
        L.qk_add_rmsnorm_q8.restype = i32
        L.qk_add_rmsnorm_q8.argtypes = [vp, i32, vp, vp, f32, vp, vp, vp, i64, i64, vp]
        L.qk_rope_kv_append.restype = i32
        L.qk_rope_kv_append.argtypes = [vp, vp, vp, vp, vp, vp, vp, i64, i64, i64, i64, i64, i64, i64, i32, f32, vp]
        L.qk_norm_rope_kv_append.restype = i32
        L.qk_norm_rope_kv_append.argtypes = [vp, vp, vp, vp, vp, f32, vp, vp, vp, vp, i64, i64, i64, i64, i64, i64, i64,
                                             i32, f32, vp]
        L.qk_norm_rope_kv_append_q4.restype = i32
        L.qk_norm_rope_kv_append_q4.argtypes = [vp, vp, vp, vp, vp, f32, vp, vp, vp, vp, vp, vp, i64, i64, i64, i64,
                                                i64, i64, i64, i32, f32, vp]
        L.qk_dequant_kv_q4.restype = i32
        L.qk_dequant_kv_q4.argtypes = [vp, vp, vp, i64, i64, i64, i64, i64, vp]
        L.qk_gqa_attention_q4.restype = i32
        L.qk_gqa_attention_q4.argtypes = [vp, vp, vp, vp, vp, vp, i64, i64, i64, i64, i64, i64, f32, i64, i64, vp, vp]
        L.qk_gqa_attention_q4_scratch_bytes.restype = i64
        L.qk_gqa_attention_q4_scratch_bytes.argtypes = [i64] * 7
        L.qk_rope_inv_freq.restype = i32
        L.qk_rope_inv_freq.argtypes = [ctypes.POINTER(qk_rope_config), i64, ctypes.POINTER(ctypes.c_double)]
        L.qk_logprobs.restype = i32
        L.qk_logprobs.argtypes = [vp, vp, vp, vp, i32, vp, vp, i64, i64, vp]
        L.qk_sample.restype = i32
        L.qk_sample.argtypes = [vp, vp, vp, vp, vp, i64, i64, f32, i32, f32, f32, vp]
        L.qk_status_string.restype, L.qk_status_string.argtypes = ctypes.c_char_p, [i32]
        L.qk_version.restype, L.qk_version.argtypes = i32, []
        _lib = L
    return _lib


# dtypes accepted for fp16 buffers (x, the SwiGLU output): fp16 itself or its bits
_F16 = ("torch.float16", "torch.uint16", "torch.int16")
_F32 = ("torch.float32",)
_F64 = ("torch.float64",)
_I8 = ("torch.int8",)
_I32 = ("torch.int32",)
_U8 = ("torch.uint8",)
_F16U8 = _F16 + _U8


_dtype_names = {}  # torch dtype -> its name: str() of a dtype takes longer than the lookup


def _buf(t, nbytes: int, what, dtypes=None) -> int:
    """The address of a buffer argument.  A raw integer address (or None) is
    passed through unchecked.  A tensor must be contiguous, of one of `dtypes`
    (any dtype if None), and hold at least `nbytes` bytes: the C ABI takes
    plain pointers and cannot see how large a buffer is.  `what` names the
    argument in the error: a string, or a format and its arguments in a tuple
    (formatted only then)."""
    if t is None:
        return 0
    if isinstance(t, int):
        return t
    if dtypes is not None:
        dtype = t.dtype
        name = _dtype_names.get(dtype)
        if name is None:
            name = _dtype_names[dtype] = str(dtype)
        if name not in dtypes:
            raise ValueError("%s: dtype %s, expected one of %s" % (_what(what), dtype, ", ".join(dtypes)))
    if not t.is_contiguous():
        raise ValueError("%s: the tensor is not contiguous" % _what(what))
    if t.nbytes < nbytes:
        raise ValueError("%s: holds %d bytes, the call needs %d" % (_what(what), t.nbytes, nbytes))
    return t.data_ptr()


def _bufs(where: str, *args) -> list:
    """The addresses of buffer arguments (tensor, bytes, dtypes, name), each checked
    as by _buf: one loop for all takes 0.1 us less for each of them."""
    out = []
    for t, nbytes, dtypes, name in args:
        try:
            if _dtype_names[t.dtype] in dtypes and t.nbytes >= nbytes and t.is_contiguous():
                out.append(t.data_ptr())
                continue
        except (AttributeError, KeyError):  # None, an address, or a dtype seen for the first time
            pass
        out.append(_buf(t, nbytes, ("%s: %s", where, name), dtypes))
    return out


def _what(what) -> str:
    return what if isinstance(what, str) else what[0] % what[1:]


def _n(v) -> int:
    v = int(v)
    return v if v > 0 else 0


def _c_int(v, where: str, name: str, most: int = (1 << 63) - 1) -> int:
    """An integer argument for a C integer whose largest value is `most`: ctypes would
    take one out of range modulo its size."""
    v = int(v)
    if -most - 1 <= v <= most:
        return v
    raise ValueError("%s: %s %d does not fit a C integer" % (where, name, v))


_INT_MAX = (1 << 31) - 1


def _size(a: int, b: int, c: int = 1) -> int:
    """a * b * c, or 0 where one of them is not positive."""
    return a * b * c if a > 0 and b > 0 and c > 0 else 0


_BLOCK_BYTES = {QK_Q4_K: 144, QK_Q6_K: 210}


def _weight_bytes(qtype, N, K) -> int:
    """Bytes of N rows of K/256 super-blocks (0 for shapes the library rejects)."""
    return _n(N) * (_n(K) // 256) * _BLOCK_BYTES.get(qtype, 0)


_raw_stream = None  # device index -> the address of torch's current stream on it
_device = None      # the current device's index


def _stream(stream) -> int:
    if stream is None:
        # torch.cuda.current_stream() builds a Stream object: 2.8 us of a call,
        # against 0.2 us for the stream's address alone.
        global _raw_stream, _device
        if _raw_stream is None:
            import torch
            torch.cuda.current_device()  # sets torch's CUDA state up
            _device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)
            _raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream",
                                  lambda device: torch.cuda.current_stream(device).cuda_stream)
        return _raw_stream(_device())
    if isinstance(stream, int):
        return stream
    return int(stream.cuda_stream)


def _check(status: int, where: str) -> None:
    if status != 0:
        raise QKError(status, where)


def qk_status_string(status: int) -> str:
    return lib().qk_status_string(int(status)).decode()


def qk_version() -> int:
    return int(lib().qk_version())


def _dequant(name, qtype, blocks, n_blocks, out, stream):
    nb = _n(n_blocks)
    w = _buf(blocks, nb * (144 if qtype == QK_Q4_K else 210), name + ": blocks")
    o = _buf(out, nb * 256 * 4, name + ": out", _F32)
    _check(getattr(lib(), name)(w, int(n_blocks), o, _stream(stream)), name)


def qk_dequant_q4k(blocks, n_blocks: int, out, stream=None) -> None:
    _dequant("qk_dequant_q4k", QK_Q4_K, blocks, n_blocks, out, stream)


def qk_dequant_q6k(blocks, n_blocks: int, out, stream=None) -> None:
    _dequant("qk_dequant_q6k", QK_Q6_K, blocks, n_blocks, out, stream)


def _matmul(name, qtype, blocks, x_f16, y, M, N, K, stream):
    w = _buf(blocks, _weight_bytes(qtype, N, K), name + ": blocks")
    x = _buf(x_f16, _n(M) * _n(K) * 2, name + ": x_f16", _F16)
    o = _buf(y, _n(M) * _n(N) * 4, name + ": y", _F32)
    _check(getattr(lib(), name)(w, x, o, int(M), int(N), int(K), _stream(stream)), name)


def qk_matmul_q4k(blocks, x_f16, y, M: int, N: int, K: int, stream=None) -> None:
    _matmul("qk_matmul_q4k", QK_Q4_K, blocks, x_f16, y, M, N, K, stream)


def qk_matmul_q6k(blocks, x_f16, y, M: int, N: int, K: int, stream=None) -> None:
    _matmul("qk_matmul_q6k", QK_Q6_K, blocks, x_f16, y, M, N, K, stream)


def qk_gateup_swiglu_q4k(gate_blocks, up_blocks, x_f16, y_f16, M: int, N_ff: int, K: int, stream=None) -> None:
    name = "qk_gateup_swiglu_q4k"
    wb = _weight_bytes(QK_Q4_K, N_ff, K)
    g = _buf(gate_blocks, wb, name + ": gate_blocks")
    u = _buf(up_blocks, wb, name + ": up_blocks")
    x = _buf(x_f16, _n(M) * _n(K) * 2, name + ": x_f16", _F16)
    o = _buf(y_f16, _n(M) * _n(N_ff) * 2, name + ": y_f16", _F16)
    _check(lib().qk_gateup_swiglu_q4k(g, u, x, o, int(M), int(N_ff), int(K), _stream(stream)), name)


def _descs(problems):
    arr = (qk_matmul_desc * max(1, len(problems)))()
    for i, p in enumerate(problems):
        qt = p["qtype"]
        qt = int(_QTYPES.get(qt, qt))
        M, N, K = int(p["M"]), int(p["N"]), int(p["K"])
        up = p.get("up_blocks")
        gu = up is not None
        wb = _weight_bytes(qt, N, K)
        arr[i] = qk_matmul_desc(qt, _buf(p["blocks"], wb, ("qk_matmul_batch[%d]: blocks", i)),
                                _buf(up, wb, ("qk_matmul_batch[%d]: up_blocks", i)),
                                _buf(p["x_f16"], _n(M) * _n(K) * 2, ("qk_matmul_batch[%d]: x_f16", i), _F16),
                                _buf(p["y"], _n(M) * _n(N) * (2 if gu else 4), ("qk_matmul_batch[%d]: y", i),
                                     _F16 if gu else _F32), M, N, K)
    return arr


def qk_matmul_batch(problems, stream=None) -> None:
    """Run independent problems in as few launches as possible.  Each problem is
    a dict with keys qtype ("q4k"/"q6k" or 0/1), blocks, x_f16, y, M, N, K and
    optionally up_blocks (fused gate/up + SwiGLU, fp16 y)."""
    arr = _descs(problems)
    _check(lib().qk_matmul_batch(arr, len(problems), _stream(stream)), "qk_matmul_batch")


def qk_matmul_batch_q8x(problems, stream=None) -> None:
    """qk_matmul_batch with int8 activations (decode only; see include/qk.h)."""
    arr = _descs(problems)
    _check(lib().qk_matmul_batch_q8x(arr, len(problems), _stream(stream)), "qk_matmul_batch_q8x")


def qk_matmul_q8x_q4k(blocks, x_f16, y, M: int, N: int, K: int, stream=None) -> None:
    """y = int8(x) . W^T for Q4_K W, M <= 1 (see include/qk.h)."""
    qk_matmul_batch_q8x([dict(qtype=QK_Q4_K, blocks=blocks, x_f16=x_f16, y=y, M=M, N=N, K=K)], stream)


def qk_matmul_q8x_q6k(blocks, x_f16, y, M: int, N: int, K: int, stream=None) -> None:
    """y = int8(x) . W^T for Q6_K W, M <= 1 (see include/qk.h)."""
    qk_matmul_batch_q8x([dict(qtype=QK_Q6_K, blocks=blocks, x_f16=x_f16, y=y, M=M, N=N, K=K)], stream)


def qk_matmul_batch_q8(problems, stream=None) -> None:
    """qk_matmul_batch_q8x for x that is in int8 already (see include/qk.h).  Each
    problem is a dict with keys qtype, blocks, x_q8 (int8 [M][K]), x_d (fp32
    [M][K / 32]), y, M, N, K and optionally up_blocks; M <= 1."""
    arr = (qk_matmul_q8_desc * max(1, len(problems)))()
    for i, p in enumerate(problems):
        qt = p["qtype"]
        qt = int(_QTYPES.get(qt, qt))
        M, N, K = int(p["M"]), int(p["N"]), int(p["K"])
        up = p.get("up_blocks")
        gu = up is not None
        wb = _size(N, K // 256, _BLOCK_BYTES.get(qt, 0))
        n = _size(M, K)
        arr[i] = qk_matmul_q8_desc(qt, _buf(p["blocks"], wb, ("qk_matmul_batch_q8[%d]: blocks", i)),
                                   _buf(up, wb, ("qk_matmul_batch_q8[%d]: up_blocks", i)),
                                   _buf(p["x_q8"], n, ("qk_matmul_batch_q8[%d]: x_q8", i), _I8),
                                   _buf(p["x_d"], n // 8, ("qk_matmul_batch_q8[%d]: x_d", i), _F32),
                                   _buf(p["y"], _size(M, N, 2 if gu else 4), ("qk_matmul_batch_q8[%d]: y", i),
                                        _F16 if gu else _F32), M, N, K)
    _check(lib().qk_matmul_batch_q8(arr, len(problems), _stream(stream)), "qk_matmul_batch_q8")


def _residual(names, residual, delta, gamma_f16, residual_out, residual_type, n, K):
    """Addresses and element type of an add_rmsnorm call's inputs and residual output."""
    if residual_type is None:
        if isinstance(residual, int) or residual is None:
            raise ValueError("%s: residual_type is needed for a raw address" % names[0])
        dtype = residual.dtype
        residual_type = QK_F32 if (_dtype_names.get(dtype) or str(dtype)) in _F32 else QK_F16
    types, size = (_F32, 4 * n) if residual_type == QK_F32 else (_F16, 2 * n)
    return (_buf(residual, size, names[0], types), int(residual_type), _buf(delta, 4 * n, names[1], _F32),
            _buf(gamma_f16, 2 * K, names[2], _F16), _buf(residual_out, size, names[3], types))


_ADD_RMSNORM = tuple("qk_add_rmsnorm: " + n for n in ("residual", "delta", "gamma_f16", "residual_out"))
_ADD_RMSNORM_Q8 = tuple("qk_add_rmsnorm_q8: " + n for n in ("residual", "delta", "gamma_f16", "residual_out"))


def qk_add_rmsnorm(residual, delta, gamma_f16, eps: float, residual_out, xhat_f16, M: int, K: int,
                   residual_type=None, stream=None) -> None:
    """h = residual + delta, residual_out = h, xhat = fp16(RMSNorm(h) * gamma) (see
    include/qk.h).  residual is fp16 or fp32 (residual_type QK_F16 / QK_F32, by
    default the tensor's own); delta and residual_out may be None."""
    k = _n(K)
    n = _n(M) * k
    r, t, d, g, o = _residual(_ADD_RMSNORM, residual, delta, gamma_f16, residual_out, residual_type, n, k)
    x = _buf(xhat_f16, 2 * n, "qk_add_rmsnorm: xhat_f16", _F16)
    _check(lib().qk_add_rmsnorm(r, t, d, g, float(eps), o, x, int(M), int(K), _stream(stream)), "qk_add_rmsnorm")


def qk_add_rmsnorm_q8(residual, delta, gamma_f16, eps: float, residual_out, xq, xd, M: int, K: int,
                      residual_type=None, stream=None) -> None:
    """qk_add_rmsnorm with the activations in int8 (xq [M][K], xd fp32 [M][K / 32]):
    the x of qk_matmul_batch_q8."""
    k = _n(K)
    n = _n(M) * k
    r, t, d, g, o = _residual(_ADD_RMSNORM_Q8, residual, delta, gamma_f16, residual_out, residual_type, n, k)
    q = _buf(xq, n, "qk_add_rmsnorm_q8: xq", _I8)
    s = _buf(xd, n // 8, "qk_add_rmsnorm_q8: xd", _F32)
    _check(lib().qk_add_rmsnorm_q8(r, t, d, g, float(eps), o, q, s, int(M), int(K), _stream(stream)),
           "qk_add_rmsnorm_q8")


def qk_rope_inv_freq(n_rot: int, theta: float, scaling: int = QK_ROPE_SCALE_NONE, factor: float = 1.0,
                     low_turns: float = 1.0, high_turns: float = 4.0, original_len: int = 8192,
                     freq_factors=None) -> list:
    """The n_rot / 2 rotation frequencies (radians per position) for
    qk_rope_kv_append's inv_freq, as Python floats; host only (see include/qk.h)."""
    half = _n(n_rot) // 2
    ff = None
    if freq_factors is not None:
        ff = [float(f) for f in freq_factors]
        if len(ff) < half:
            raise ValueError("qk_rope_inv_freq: %d freq_factors, n_rot %d needs %d" % (len(ff), n_rot, half))
        ff = (ctypes.c_float * max(1, len(ff)))(*ff)
    cfg = qk_rope_config(float(theta), int(scaling), float(factor), float(low_turns), float(high_turns),
                         int(original_len), ff)
    out = (ctypes.c_double * max(1, half))()
    _check(lib().qk_rope_inv_freq(ctypes.byref(cfg), int(n_rot), out), "qk_rope_inv_freq")
    return list(out[:half])


def qk_rope_kv_append(q, k, v, inv_freq, q_f16, k_cache, v_cache, M: int, H: int, H_kv: int, D: int, n_rot: int,
                      pos0: int, L_max: int, layout: int = QK_ROPE_INTERLEAVED, magnitude: float = 1.0,
                      stream=None) -> None:
    """Rotary positions on the QKV projections' outputs and the new cache rows (see
    include/qk.h): q, k, v fp32 [M][heads][D], inv_freq float64 [n_rot / 2], q_f16
    [M][H][D] fp16, caches [H_kv][L_max][D] fp16."""
    M, H, H_kv, D, L_max = int(M), int(H), int(H_kv), int(D), int(L_max)
    qn, kn, cn = _size(M, H, D), _size(M, H_kv, D), _size(H_kv, L_max, D)
    _check(lib().qk_rope_kv_append(_buf(q, 4 * qn, "qk_rope_kv_append: q", _F32), _buf(k, 4 * kn, "qk_rope_kv_append: k", _F32),
                                   _buf(v, 4 * kn, "qk_rope_kv_append: v", _F32),
                                   _buf(inv_freq, 4 * _n(n_rot), "qk_rope_kv_append: inv_freq", _F64),
                                   _buf(q_f16, 2 * qn, "qk_rope_kv_append: q_f16", _F16),
                                   _buf(k_cache, 2 * cn, "qk_rope_kv_append: k_cache", _F16),
                                   _buf(v_cache, 2 * cn, "qk_rope_kv_append: v_cache", _F16), M, H, H_kv, D,
                                   int(n_rot), _c_int(pos0, "qk_rope_kv_append", "pos0"), L_max,
                                   _c_int(layout, "qk_rope_kv_append", "layout", _INT_MAX), float(magnitude),
                                   _stream(stream)), "qk_rope_kv_append")


def qk_norm_rope_kv_append(q, k, v, q_gamma_f16, k_gamma_f16, eps: float, inv_freq, q_f16, k_cache, v_cache, M: int,
                           H: int, H_kv: int, D: int, n_rot: int, pos0: int, L_max: int,
                           layout: int = QK_ROPE_INTERLEAVED, magnitude: float = 1.0, stream=None) -> None:
    """qk_rope_kv_append with an RMSNorm of each query and key head in front (see
    include/qk.h): gammas fp16 [D], or None for heads that are not normalized."""
    M, H, H_kv, D, n_rot, L_max = int(M), int(H), int(H_kv), int(D), int(n_rot), int(L_max)
    cn = 2 * _size(H_kv, L_max, D)
    pos0, layout = _append_ints("qk_norm_rope_kv_append", pos0, layout)
    a = _bufs("qk_norm_rope_kv_append",
              *_append_args(q, k, v, q_gamma_f16, k_gamma_f16, inv_freq, q_f16, M, H, H_kv, D, n_rot),
              (k_cache, cn, _F16, "k_cache"), (v_cache, cn, _F16, "v_cache"))
    _check(lib().qk_norm_rope_kv_append(a[0], a[1], a[2], a[3], a[4], float(eps), a[5], a[6], a[7], a[8], M, H, H_kv, D,
                                        n_rot, pos0, L_max, layout, float(magnitude), _stream(stream)),
           "qk_norm_rope_kv_append")


def _append_ints(where, pos0, layout):
    return _c_int(pos0, where, "pos0"), _c_int(layout, where, "layout", _INT_MAX)


def _append_args(q, k, v, q_gamma_f16, k_gamma_f16, inv_freq, q_f16, M, H, H_kv, D, n_rot):
    qn, kn, gn = _size(M, H, D), 4 * _size(M, H_kv, D), 2 * D
    return ((q, 4 * qn, _F32, "q"), (k, kn, _F32, "k"), (v, kn, _F32, "v"), (q_gamma_f16, gn, _F16, "q_gamma_f16"),
            (k_gamma_f16, gn, _F16, "k_gamma_f16"), (inv_freq, 4 * n_rot, _F64, "inv_freq"),
            (q_f16, 2 * qn, _F16, "q_f16"))


def qk_norm_rope_kv_append_q4(q, k, v, q_gamma_f16, k_gamma_f16, eps: float, inv_freq, q_f16, k_q4, k_dm, v_q4, v_dm,
                              M: int, H: int, H_kv: int, D: int, n_rot: int, pos0: int, L_max: int,
                              layout: int = QK_ROPE_INTERLEAVED, magnitude: float = 1.0, stream=None) -> None:
    """qk_norm_rope_kv_append into a cache held in 4 bits (see include/qk.h): k_q4, v_q4
    uint8 [H_kv][L_max][D / 2], k_dm, v_dm fp16 [H_kv][L_max][D / 32][2]."""
    M, H, H_kv, D, n_rot, L_max = int(M), int(H), int(H_kv), int(D), int(n_rot), int(L_max)
    cn = _size(H_kv, L_max, D)
    pos0, layout = _append_ints("qk_norm_rope_kv_append_q4", pos0, layout)
    a = _bufs("qk_norm_rope_kv_append_q4",
              *_append_args(q, k, v, q_gamma_f16, k_gamma_f16, inv_freq, q_f16, M, H, H_kv, D, n_rot),
              (k_q4, cn // 2, _U8, "k_q4"), (k_dm, cn // 8, _F16, "k_dm"), (v_q4, cn // 2, _U8, "v_q4"),
              (v_dm, cn // 8, _F16, "v_dm"))
    _check(lib().qk_norm_rope_kv_append_q4(a[0], a[1], a[2], a[3], a[4], float(eps), a[5], a[6], a[7], a[8], a[9], a[10],
                                           M, H, H_kv, D, n_rot, pos0, L_max, layout, float(magnitude),
                                           _stream(stream)), "qk_norm_rope_kv_append_q4")


def qk_dequant_kv_q4(q4, dm, out_f16, H_kv: int, D: int, pos0: int, M: int, L_max: int, stream=None) -> None:
    """Rows pos0 .. pos0 + M - 1 of one tensor of a 4-bit cache as fp16 [H_kv][M][D] (see include/qk.h)."""
    H_kv, D, M, L_max = int(H_kv), int(D), int(M), int(L_max)
    cn = _size(H_kv, L_max, D)
    a = _bufs("qk_dequant_kv_q4", (q4, cn // 2, _U8, "q4"), (dm, cn // 8, _F16, "dm"),
              (out_f16, 2 * _size(H_kv, M, D), _F16, "out_f16"))
    _check(lib().qk_dequant_kv_q4(a[0], a[1], a[2], H_kv, D, _c_int(pos0, "qk_dequant_kv_q4", "pos0"), M, L_max,
                                  _stream(stream)), "qk_dequant_kv_q4")


def qk_rmsnorm_scratch_bytes(qtype, M: int, K: int, gateup: bool = False) -> int:
    """Scratch bytes an M-token problem needs under the RMSNorm entry points
    (0 when the GEMV fuses the norm); host only."""
    qt = {"q4k": QK_Q4_K, "q6k": QK_Q6_K}.get(qtype, qtype)
    r = int(lib().qk_rmsnorm_scratch_bytes(int(qt), int(bool(gateup)), int(M), int(K)))
    if r < 0:
        raise ValueError("qk_rmsnorm_scratch_bytes: invalid qtype %r, M %d or K %d" % (qtype, M, K))
    return r


def _scratch(problems, scratch, what):
    need = 0
    for p in problems:
        qt = {"q4k": QK_Q4_K, "q6k": QK_Q6_K}.get(p["qtype"], p["qtype"])
        if int(p["M"]) > 0 and int(p["N"]) > 0:
            need = max(need, qk_rmsnorm_scratch_bytes(qt, p["M"], p["K"], p.get("up_blocks") is not None))
    return _buf(scratch, need, what + ": scratch", _F16 + ("torch.uint8",))


def qk_rmsnorm_matmul_batch(problems, gamma_f16, eps: float, scratch=None, stream=None) -> None:
    """qk_matmul_batch over RMSNorm(x) * gamma (see include/qk.h); `scratch` is
    needed for problems the tensor-core GEMM runs (qk_rmsnorm_scratch_bytes)."""
    what = "qk_rmsnorm_matmul_batch"
    arr = _descs(problems)
    K = max([int(p["K"]) for p in problems] or [0])
    g = _buf(gamma_f16, 2 * K, what + ": gamma_f16", _F16)
    sc = _scratch(problems, scratch, what)
    _check(lib().qk_rmsnorm_matmul_batch(arr, len(problems), g, float(eps), sc, _stream(stream)), what)


def qk_rmsnorm_matmul_batch_static(problems, gamma_f16, eps: float, stream=None) -> None:
    """qk_rmsnorm_matmul_batch for callers that cannot allocate device memory
    (a CUDA graph being captured, a framework whose pool owns the GPU, a loop
    that must not block in cudaMalloc): the scratch is a fixed 8 MiB array in
    the library, shared by every call, so calls that may overlap on the GPU
    race on it.  Problems needing more scratch raise QKError (QK_ERR_SCRATCH)."""
    what = "qk_rmsnorm_matmul_batch_static"
    arr = _descs(problems)
    K = max([int(p["K"]) for p in problems] or [0])
    g = _buf(gamma_f16, 2 * K, what + ": gamma_f16", _F16)
    _check(lib().qk_rmsnorm_matmul_batch_static(arr, len(problems), g, float(eps), _stream(stream)), what)


def _rms_single(name, qtype, blocks, up_blocks, x_f16, gamma_f16, eps, scratch, y, M, N, K, stream):
    gu = up_blocks is not None
    wb = _weight_bytes(qtype, N, K)
    w = _buf(blocks, wb, name + ": blocks")
    x = _buf(x_f16, _n(M) * _n(K) * 2, name + ": x_f16", _F16)
    g = _buf(gamma_f16, 2 * _n(K), name + ": gamma_f16", _F16)
    need = qk_rmsnorm_scratch_bytes(qtype, max(0, int(M)), K, gu) if int(K) > 0 and int(K) % 256 == 0 else 0
    sc = _buf(scratch, need, name + ": scratch", _F16 + ("torch.uint8",))
    if gu:
        u = _buf(up_blocks, wb, name + ": up_blocks")
        o = _buf(y, _n(M) * _n(N) * 2, name + ": y_f16", _F16)
        rc = lib().qk_rmsnorm_gateup_swiglu_q4k(w, u, x, g, float(eps), sc, o, int(M), int(N), int(K), _stream(stream))
    else:
        o = _buf(y, _n(M) * _n(N) * 4, name + ": y", _F32)
        rc = getattr(lib(), name)(w, x, g, float(eps), sc, o, int(M), int(N), int(K), _stream(stream))
    _check(rc, name)


def qk_rmsnorm_matmul_q4k(blocks, x_f16, gamma_f16, eps, y, M, N, K, scratch=None, stream=None) -> None:
    _rms_single("qk_rmsnorm_matmul_q4k", QK_Q4_K, blocks, None, x_f16, gamma_f16, eps, scratch, y, M, N, K, stream)


def qk_rmsnorm_matmul_q6k(blocks, x_f16, gamma_f16, eps, y, M, N, K, scratch=None, stream=None) -> None:
    _rms_single("qk_rmsnorm_matmul_q6k", QK_Q6_K, blocks, None, x_f16, gamma_f16, eps, scratch, y, M, N, K, stream)


def qk_rmsnorm_gateup_swiglu_q4k(gate_blocks, up_blocks, x_f16, gamma_f16, eps, y_f16, M, N_ff, K, scratch=None,
                                 stream=None) -> None:
    _rms_single("qk_rmsnorm_gateup_swiglu_q4k", QK_Q4_K, gate_blocks, up_blocks, x_f16, gamma_f16, eps, scratch,
                y_f16, M, N_ff, K, stream)


def qk_decode_uses_gemv(qtype, K: int, gateup: bool = False) -> bool:
    """Whether an M = 1 problem of this format and K runs on the decode GEMV
    (True) or on the tensor-core GEMM (False); host only."""
    qt = {"q4k": QK_Q4_K, "q6k": QK_Q6_K}.get(qtype, qtype)
    r = int(lib().qk_decode_uses_gemv(int(qt), int(bool(gateup)), int(K)))
    if r < 0:
        raise ValueError("qk_decode_uses_gemv: invalid qtype %r or K %d" % (qtype, K))
    return bool(r)


def qk_uses_gemv(qtype, M: int, K: int, gateup: bool = False) -> bool:
    """Whether an M-token problem of this format and K runs on the GEMV (True)
    or on the tensor-core GEMM (False); host only."""
    qt = {"q4k": QK_Q4_K, "q6k": QK_Q6_K}.get(qtype, qtype)
    r = int(lib().qk_uses_gemv(int(qt), int(bool(gateup)), int(M), int(K)))
    if r < 0:
        raise ValueError("qk_uses_gemv: invalid qtype %r, M %d or K %d" % (qtype, M, K))
    return bool(r)


def qk_gemm_plan(qtype, M: int, N: int, K: int, gateup: bool = False) -> dict:
    """The tensor-core GEMM's launch plan for an M x N x K problem (host only)."""
    qt = {"q4k": QK_Q4_K, "q6k": QK_Q6_K}.get(qtype, qtype)
    info = qk_gemm_plan_info()
    _check(lib().qk_gemm_plan(int(qt), int(bool(gateup)), int(M), int(N), int(K), ctypes.byref(info)),
           "qk_gemm_plan")
    return {n: getattr(info, n) for n, _ in qk_gemm_plan_info._fields_}


def qk_gqa_attention(q_f16, k_cache, v_cache, out, M: int, H: int, H_kv: int, D: int, pos0: int, L_max: int,
                     scale: float, stream=None) -> None:
    """GQA attention over a KV cache (see include/qk.h): q [M][H][D] fp16,
    caches [H_kv][L_max][D] fp16, out [M][H][D] fp32."""
    what = "qk_gqa_attention"
    qn = _n(M) * _n(H) * _n(D)
    cn = _n(H_kv) * _n(L_max) * _n(D)
    _check(lib().qk_gqa_attention(_buf(q_f16, 2 * qn, what + ": q_f16", _F16),
                                  _buf(k_cache, 2 * cn, what + ": k_cache", _F16),
                                  _buf(v_cache, 2 * cn, what + ": v_cache", _F16),
                                  _buf(out, 4 * qn, what + ": out", _F32), int(M), int(H), int(H_kv), int(D),
                                  _c_int(pos0, what, "pos0"), int(L_max), float(scale), _stream(stream)), what)


def qk_gqa_attention_window(q_f16, k_cache, v_cache, out_f16, M: int, H: int, H_kv: int, D: int, pos0: int,
                            L_max: int, scale: float, window: int, sinks: int = 0, stream=None) -> None:
    """qk_gqa_attention with a sliding window of `window` positions and the first
    `sinks` positions always visible (see include/qk.h); out [M][H][D] fp16."""
    M, H, H_kv, D, L_max = int(M), int(H), int(H_kv), int(D), int(L_max)
    pos0, window, sinks = _window_ints("qk_gqa_attention_window", pos0, window, sinks)
    qn, cn = _size(M, H, D), _size(H_kv, L_max, D)
    _check(lib().qk_gqa_attention_window(_buf(q_f16, 2 * qn, "qk_gqa_attention_window: q_f16", _F16),
                                         _buf(k_cache, 2 * cn, "qk_gqa_attention_window: k_cache", _F16),
                                         _buf(v_cache, 2 * cn, "qk_gqa_attention_window: v_cache", _F16),
                                         _buf(out_f16, 2 * qn, "qk_gqa_attention_window: out_f16", _F16), M, H, H_kv,
                                         D, pos0, L_max, float(scale), window, sinks, _stream(stream)),
           "qk_gqa_attention_window")


def _window_ints(where, pos0, window, sinks):
    return _c_int(pos0, where, "pos0"), _c_int(window, where, "window"), _c_int(sinks, where, "sinks")


def qk_gqa_attention_q4_scratch_bytes(M: int, H: int, H_kv: int, D: int, pos0: int, window: int, sinks: int = 0) -> int:
    """Scratch bytes that qk_gqa_attention_q4 needs (0: none); host only."""
    where = "qk_gqa_attention_q4_scratch_bytes"
    M, H, H_kv, D = (_c_int(v, where, "size") for v in (M, H, H_kv, D))
    r = int(lib().qk_gqa_attention_q4_scratch_bytes(M, H, H_kv, D, *_window_ints(where, pos0, window, sinks)))
    if r < 0:
        raise ValueError("qk_gqa_attention_q4_scratch_bytes: invalid sizes")
    return r


def qk_gqa_attention_q4(q_f16, k_q4, k_dm, v_q4, v_dm, out_f16, M: int, H: int, H_kv: int, D: int, pos0: int,
                        L_max: int, scale: float, window: int, sinks: int = 0, scratch=None, stream=None) -> None:
    """qk_gqa_attention_window over a cache held in 4 bits (see include/qk.h); scratch:
    qk_gqa_attention_q4_scratch_bytes of device memory where that is not 0."""
    M, H, H_kv, D, L_max = int(M), int(H), int(H_kv), int(D), int(L_max)
    pos0, window, sinks = _window_ints("qk_gqa_attention_q4", pos0, window, sinks)
    qn, cn = _size(M, H, D), _size(H_kv, L_max, D)
    # fp16 rows of all positions are as much as any call needs: no need to ask then
    need = 0
    if scratch is not None and not isinstance(scratch, int) and scratch.nbytes < 512 * H_kv * (pos0 + M):
        need = max(0, lib().qk_gqa_attention_q4_scratch_bytes(M, H, H_kv, D, pos0, window, sinks))
    a = _bufs("qk_gqa_attention_q4", (q_f16, 2 * qn, _F16, "q_f16"), (k_q4, cn // 2, _U8, "k_q4"),
              (k_dm, cn // 8, _F16, "k_dm"), (v_q4, cn // 2, _U8, "v_q4"), (v_dm, cn // 8, _F16, "v_dm"),
              (out_f16, 2 * qn, _F16, "out_f16"), (scratch, need, _F16U8, "scratch"))
    _check(lib().qk_gqa_attention_q4(a[0], a[1], a[2], a[3], a[4], a[5], M, H, H_kv, D, pos0, L_max, float(scale),
                                     window, sinks, a[6], _stream(stream)), "qk_gqa_attention_q4")


def qk_logprobs(logits, tokens, logprob, entropy, top_n: int, top_ids, top_logprobs, M: int, V: int,
                stream=None) -> None:
    """Log probabilities of given tokens, entropy and the top_n alternatives of each
    row of logits fp32 [M][V] (see include/qk.h): tokens int32 [M], logprob and
    entropy fp32 [M], top_ids int32 and top_logprobs fp32 [M][top_n].  tokens and
    logprob may both be None, so may entropy, and top_ids and top_logprobs for
    top_n = 0."""
    m = 4 * _n(M)
    _check(lib().qk_logprobs(_buf(logits, m * _n(V), "qk_logprobs: logits", _F32),
                             _buf(tokens, m, "qk_logprobs: tokens", _I32), _buf(logprob, m, "qk_logprobs: logprob", _F32),
                             _buf(entropy, m, "qk_logprobs: entropy", _F32),
                             _c_int(top_n, "qk_logprobs", "top_n", _INT_MAX),
                             _buf(top_ids, m * _n(top_n), "qk_logprobs: top_ids", _I32),
                             _buf(top_logprobs, m * _n(top_n), "qk_logprobs: top_logprobs", _F32), int(M), int(V),
                             _stream(stream)), "qk_logprobs")


def qk_sample(logits, u, token, logprob, kept, M: int, V: int, temperature: float = 1.0, top_k: int = 0,
              top_p: float = 1.0, min_p: float = 0.0, stream=None) -> None:
    """A token from each row of logits fp32 [M][V] and a given random number u fp32 [M]
    (see include/qk.h): token int32 [M], logprob fp32 [M] and kept int32 [M] or None."""
    M, V = int(M), int(V)
    m = 4 * _n(M)
    a = _bufs("qk_sample", (logits, m * _n(V), _F32, "logits"), (u, m, _F32, "u"), (token, m, _I32, "token"),
              (logprob, m, _F32, "logprob"), (kept, m, _I32, "kept"))
    _check(lib().qk_sample(a[0], a[1], a[2], a[3], a[4], M, V, float(temperature),
                           _c_int(top_k, "qk_sample", "top_k", _INT_MAX), float(top_p), float(min_p), _stream(stream)),
           "qk_sample")


def qk_get_device_status(stream=None) -> None:
    _check(lib().qk_get_device_status(_stream(stream)), "qk_get_device_status")


def qk_debug_wait_timeout(limit_ns: int, stream=None) -> None:
    """Enqueue a kernel whose only wait times out after ``limit_ns`` (see include/qk.h)."""
    _check(lib().qk_debug_wait_timeout(int(limit_ns), _stream(stream)), "qk_debug_wait_timeout")
