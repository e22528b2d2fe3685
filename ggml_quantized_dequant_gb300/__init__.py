"""Python binding of the qdq CUDA library (libqdq.so): argument marshalling only.

Every function here takes torch CUDA tensors (or raw device pointers as ints),
passes their addresses, sizes and the current CUDA stream to the C ABI declared
in ``include/qdq.h``, and raises :class:`QdqError` on a non-zero status.  All
arithmetic runs in the CUDA kernels; there is no CPU path.  The library is
built in-tree by ``__graft_entry__.build()`` (or ``python -m
ggml_quantized_dequant_gb300._build``); loading fails loudly if it is absent.
"""
from __future__ import annotations

import ctypes
import os

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libqdq.so")

QDQ_OK = 0
QDQ_ERR_NULL = -1
QDQ_ERR_DIMS = -2
QDQ_ERR_ALIGN = -3
QDQ_ERR_UNSUPPORTED = -4
QDQ_ERR_CUDA = -5
QDQ_ERR_ALIAS = -6
QDQ_ERR_SCRATCH = -7
QDQ_NOALLOC_FFN_MAX_MID = 262144
QDQ_MAX_GEMV_BATCH = 8
QDQ_MAX_TOPK = 64
QDQ_MAX_GEMV_N_IN = 32768
QDQ_MAX_NORM_N = 32768
QDQ_KV_BLOCK = 16
QDQ_MAX_KV_LEN = 4194304
QDQ_TYPE_F32 = 0
QDQ_TYPE_F16 = 1
QDQ_TYPE_BF16 = 2
QDQ_OPT_PDL = 1
QDQ_OPT_L2_PREFETCH = 2
QDQ_OPT_CTAS_PER_SM = 3
QDQ_OPT_XS_GROUPS = 4
QDQ_OPT_XS_STAGES = 5
QDQ_OPT_XS_FLOAT_X = 6
QDQ_OPT_BATCH1_KERNEL = 7
QDQ_OPT_ATTN_KERNEL = 8

_c_int, _c_size, _c_vp, _c_char_p = ctypes.c_int, ctypes.c_size_t, ctypes.c_void_p, ctypes.c_char_p
_c_ll, _c_float = ctypes.c_longlong, ctypes.c_float

# name -> (restype, argtypes); mirrors include/qdq.h
SIGNATURES = {
    "qdq_status_string": (_c_char_p, [_c_int]),
    "qdq_last_cuda_error": (_c_int, []),
    "qdq_version": (_c_char_p, []),
    "qdq_q8_0_packed_bytes": (_c_size, [_c_int, _c_int]),
    "qdq_q4k_packed_bytes": (_c_size, [_c_int, _c_int]),
    "qdq_q8_0_pack": (_c_int, [_c_vp, _c_vp, _c_int, _c_int, _c_vp]),
    "qdq_q4k_pack": (_c_int, [_c_vp, _c_vp, _c_int, _c_int, _c_vp]),
    "qdq_q8_0_dequant": (_c_int, [_c_vp, _c_vp, _c_int, _c_int, _c_vp]),
    "qdq_q4k_dequant": (_c_int, [_c_vp, _c_vp, _c_int, _c_int, _c_vp]),
    "qdq_q8_0_gemv": (_c_int, [_c_vp, _c_vp, _c_vp, _c_int, _c_int, _c_int, _c_vp]),
    "qdq_q4k_gemv": (_c_int, [_c_vp, _c_vp, _c_vp, _c_int, _c_int, _c_int, _c_vp]),
    "qdq_q4k_swiglu": (_c_int, [_c_vp, _c_vp, _c_vp, _c_vp, _c_int, _c_int, _c_int, _c_vp]),
    "qdq_q8_0_logits_argmax": (_c_int, [_c_vp, _c_vp, _c_vp, _c_vp, _c_vp, _c_int, _c_int, _c_int, _c_vp]),
    "qdq_q4k_qkv": (_c_int, [_c_vp, _c_vp, _c_vp, _c_vp, _c_vp, _c_vp, _c_vp, _c_int, _c_int, _c_int, _c_int,
                             _c_vp]),
    "qdq_q4k_ffn_residual": (_c_int, [_c_vp, _c_vp, _c_vp, _c_vp, _c_vp, _c_vp, _c_vp,
                                      _c_int, _c_int, _c_int, _c_vp]),
    "qdq_q4k_ffn_residual_noalloc": (_c_int, [_c_vp, _c_vp, _c_vp, _c_vp, _c_vp, _c_vp,
                                              _c_int, _c_int, _c_int, _c_vp]),
    "qdq_q6k_packed_bytes": (_c_size, [_c_int, _c_int]),
    "qdq_q6k_pack": (_c_int, [_c_vp, _c_vp, _c_int, _c_int, _c_vp]),
    "qdq_q6k_dequant": (_c_int, [_c_vp, _c_vp, _c_int, _c_int, _c_vp]),
    "qdq_q6k_gemv": (_c_int, [_c_vp, _c_vp, _c_vp, _c_int, _c_int, _c_int, _c_vp]),
    "qdq_q6k_get_rows": (_c_int, [_c_vp, _c_vp, _c_vp, _c_int, _c_int, _c_int, _c_vp]),
    "qdq_topk_workspace_bytes": (_c_size, [_c_int, _c_int, _c_int]),
    "qdq_topk_rows": (_c_int, [_c_vp, _c_int, _c_int, _c_int, _c_vp, _c_vp, _c_vp, _c_vp]),
    "qdq_q8_0_logits_topk": (_c_int, [_c_vp, _c_vp, _c_vp, _c_vp, _c_vp, _c_vp, _c_int, _c_int, _c_int, _c_int,
                                      _c_vp]),
    "qdq_gemm_batch_workspace_bytes": (_c_size, [_c_int, _c_int, _c_int]),
    "qdq_q8_0_gemm_batch": (_c_int, [_c_vp, _c_vp, _c_vp, _c_vp, _c_int, _c_int, _c_int, _c_vp]),
    "qdq_q4k_gemm_batch": (_c_int, [_c_vp, _c_vp, _c_vp, _c_vp, _c_int, _c_int, _c_int, _c_vp]),
    "qdq_q4k_swiglu_batch_workspace_bytes": (_c_size, [_c_int, _c_int, _c_int]),
    "qdq_q4k_swiglu_batch": (_c_int, [_c_vp, _c_vp, _c_vp, _c_vp, _c_vp, _c_int, _c_int, _c_int, _c_vp]),
    "qdq_rms_norm": (_c_int, [_c_vp] * 6 + [_c_int] * 3 + [_c_ll] * 4 + [_c_float, _c_vp]),
    "qdq_kv_page_bytes": (_c_size, [_c_int, _c_int, _c_int]),
    "qdq_kv_append": (_c_int, [_c_vp] + [_c_int] * 4 + [_c_vp, _c_int, _c_vp, _c_vp, _c_int, _c_int, _c_vp, _c_vp, _c_ll,
                               _c_ll, _c_int, _c_vp]),
    "qdq_kv_read": (_c_int, [_c_vp] + [_c_int] * 4 + [_c_vp, _c_int, _c_vp, _c_vp, _c_int, _c_int, _c_vp, _c_vp, _c_ll,
                             _c_ll, _c_int, _c_vp]),
    "qdq_kv_attention_workspace_bytes": (_c_size, [_c_int] * 6),
    "qdq_kv_attention": (_c_int, [_c_vp] + [_c_int] * 4 + [_c_vp, _c_int, _c_vp, _c_vp] + [_c_int] * 4
                         + [_c_vp, _c_ll, _c_vp, _c_ll, _c_vp, _c_vp, _c_float, _c_float, _c_int, _c_int, _c_vp, _c_size,
                            _c_vp]),
    "qdq_token_logprobs_workspace_bytes": (_c_size, [_c_int] * 3),
    "qdq_token_logprobs": (_c_int, [_c_vp, _c_ll, _c_int, _c_vp, _c_int, _c_int, _c_int] + [_c_vp] * 5 + [_c_size, _c_vp]),
    "qdq_pipeline_timeouts": (_c_int, []),
    "qdq_noop": (_c_int, [_c_vp]),
    "qdq_check_status": (_c_int, []),
    "qdq_checks_enabled": (_c_int, []),
    "qdq_set_option": (_c_int, [_c_int, _c_int]),
}

_lib = None


class QdqError(RuntimeError):
    def __init__(self, fn: str, status: int):
        self.status = status
        msg = "%s failed: %s" % (fn, status_string(status))
        if status == QDQ_ERR_CUDA and _lib is not None:
            msg += " (cudaError %d)" % _lib.qdq_last_cuda_error()
        super().__init__(msg)


def load(path: str | None = None) -> ctypes.CDLL:
    """Load libqdq.so (once) and declare every entry point's signature."""
    global _lib
    if _lib is not None:
        return _lib
    p = path or LIB_PATH
    if not os.path.exists(p):
        raise RuntimeError("libqdq.so is not built (%s); run __graft_entry__.build()" % p)
    lib = ctypes.CDLL(p)
    for name, (res, args) in SIGNATURES.items():
        fn = getattr(lib, name)
        fn.restype = res
        fn.argtypes = args
    _lib = lib
    return lib


def lib() -> ctypes.CDLL:
    return load()


def status_string(status: int) -> str:
    if _lib is None:
        return str(status)
    return _lib.qdq_status_string(int(status)).decode()


def _ptr(t) -> int | None:
    if t is None:
        return None
    if isinstance(t, int):
        return t
    return int(t.data_ptr())


def _find_current_stream() -> int:
    """The current stream of the current device; the first call binds the cheapest way to ask for it."""
    global _current_stream
    import torch
    found = int(torch.cuda.current_stream().cuda_stream)  # also initialises CUDA in torch
    try:  # the raw handle, without a Stream object for each call (3 us of a call's 6)
        get, device = torch._C._cuda_getCurrentRawStream, torch._C._cuda_getDevice
        if get(device()) == found:
            _current_stream = lambda: get(device())  # noqa: E731
    except AttributeError:
        _current_stream = lambda: int(torch.cuda.current_stream().cuda_stream)  # noqa: E731
    return found


_current_stream = _find_current_stream


def _stream(stream) -> int | None:
    if stream is None:
        return _current_stream() or None
    if isinstance(stream, int):
        return stream or None
    return int(stream.cuda_stream) or None


def _check(name: str, status: int):
    if status != QDQ_OK:
        raise QdqError(name, status)


# ---------------------------------------------------------------- C-ABI mirrors

def q8_0_packed_bytes(n_out: int, n_in: int) -> int:
    return int(lib().qdq_q8_0_packed_bytes(n_out, n_in))


def q4k_packed_bytes(n_out: int, n_in: int) -> int:
    return int(lib().qdq_q4k_packed_bytes(n_out, n_in))


def q8_0_pack(ggml, packed, n_out: int, n_in: int, stream=None):
    _check("qdq_q8_0_pack", lib().qdq_q8_0_pack(_ptr(ggml), _ptr(packed), n_out, n_in, _stream(stream)))


def q4k_pack(ggml, packed, n_out: int, n_in: int, stream=None):
    _check("qdq_q4k_pack", lib().qdq_q4k_pack(_ptr(ggml), _ptr(packed), n_out, n_in, _stream(stream)))


def q8_0_dequant(W, out, n_out: int, n_in: int, stream=None):
    _check("qdq_q8_0_dequant", lib().qdq_q8_0_dequant(_ptr(W), _ptr(out), n_out, n_in, _stream(stream)))


def q4k_dequant(W, out, n_out: int, n_in: int, stream=None):
    _check("qdq_q4k_dequant", lib().qdq_q4k_dequant(_ptr(W), _ptr(out), n_out, n_in, _stream(stream)))


def q8_0_gemv(W, x, y, n_out: int, n_in: int, batch: int = 1, stream=None):
    _check("qdq_q8_0_gemv", lib().qdq_q8_0_gemv(_ptr(W), _ptr(x), _ptr(y), n_out, n_in, batch, _stream(stream)))


def q4k_gemv(W, x, y, n_out: int, n_in: int, batch: int = 1, stream=None):
    _check("qdq_q4k_gemv", lib().qdq_q4k_gemv(_ptr(W), _ptr(x), _ptr(y), n_out, n_in, batch, _stream(stream)))


def q4k_swiglu(Wg, Wu, x, mid, n_ff: int, n_embd: int, batch: int = 1, stream=None):
    _check("qdq_q4k_swiglu", lib().qdq_q4k_swiglu(_ptr(Wg), _ptr(Wu), _ptr(x), _ptr(mid), n_ff, n_embd, batch,
                                                  _stream(stream)))


def q8_0_logits_argmax(W, x, logits, index, value, n_vocab: int, n_in: int, batch: int = 1, stream=None):
    """Output projection plus on-device argmax: ``index`` (int32) and ``value`` (f32) per batch row."""
    _check("qdq_q8_0_logits_argmax",
           lib().qdq_q8_0_logits_argmax(_ptr(W), _ptr(x), _ptr(logits), _ptr(index), _ptr(value), n_vocab, n_in,
                                        batch, _stream(stream)))


def q4k_qkv(Wq, Wk, Wv, x, q, k, v, n_q: int, n_kv: int, n_embd: int, batch: int = 1, stream=None):
    _check("qdq_q4k_qkv", lib().qdq_q4k_qkv(_ptr(Wq), _ptr(Wk), _ptr(Wv), _ptr(x), _ptr(q), _ptr(k), _ptr(v),
                                            n_q, n_kv, n_embd, batch, _stream(stream)))


def q4k_ffn_residual(Wg, Wu, Wd, x, residual, out, mid_workspace, n_embd: int, n_ff: int, batch: int = 1,
                     stream=None):
    _check("qdq_q4k_ffn_residual",
           lib().qdq_q4k_ffn_residual(_ptr(Wg), _ptr(Wu), _ptr(Wd), _ptr(x), _ptr(residual), _ptr(out),
                                      _ptr(mid_workspace), n_embd, n_ff, batch, _stream(stream)))


def q4k_ffn_residual_noalloc(Wg, Wu, Wd, x, residual, out, n_embd: int, n_ff: int, batch: int = 1, stream=None):
    """The FFN block with its intermediate vector in the library's fixed device array (no allocation).

    For callers that may not allocate device memory.  batch * n_ff must not exceed
    QDQ_NOALLOC_FFN_MAX_MID; calls that overlap on the GPU share the array and race.
    """
    _check("qdq_q4k_ffn_residual_noalloc",
           lib().qdq_q4k_ffn_residual_noalloc(_ptr(Wg), _ptr(Wu), _ptr(Wd), _ptr(x), _ptr(residual), _ptr(out),
                                              n_embd, n_ff, batch, _stream(stream)))


def q6k_packed_bytes(n_out: int, n_in: int) -> int:
    return int(lib().qdq_q6k_packed_bytes(n_out, n_in))


def q6k_pack(ggml, packed, n_out: int, n_in: int, stream=None):
    _check("qdq_q6k_pack", lib().qdq_q6k_pack(_ptr(ggml), _ptr(packed), n_out, n_in, _stream(stream)))


def q6k_dequant(W, out, n_out: int, n_in: int, stream=None):
    _check("qdq_q6k_dequant", lib().qdq_q6k_dequant(_ptr(W), _ptr(out), n_out, n_in, _stream(stream)))


def q6k_gemv(W, x, y, n_out: int, n_in: int, batch: int = 1, stream=None):
    _check("qdq_q6k_gemv", lib().qdq_q6k_gemv(_ptr(W), _ptr(x), _ptr(y), n_out, n_in, batch, _stream(stream)))


def q6k_get_rows(W, ids, out, n_ids: int, n_rows: int, n_in: int, stream=None):
    """Embedding lookup: ``out[i] = dequantised row ids[i]`` (int32 ids on the device)."""
    _check("qdq_q6k_get_rows", lib().qdq_q6k_get_rows(_ptr(W), _ptr(ids), _ptr(out), n_ids, n_rows, n_in,
                                                      _stream(stream)))


def topk_workspace_bytes(n: int, batch: int, k: int) -> int:
    return int(lib().qdq_topk_workspace_bytes(n, batch, k))


def topk_rows(logits, n: int, batch: int, k: int, workspace, index, value, stream=None):
    """Per row of ``logits``: the k best (index, value) pairs, NaN first, larger first, smaller index on ties."""
    _check("qdq_topk_rows", lib().qdq_topk_rows(_ptr(logits), n, batch, k, _ptr(workspace), _ptr(index), _ptr(value),
                                                _stream(stream)))


def q8_0_logits_topk(W, x, logits, workspace, index, value, n_vocab: int, n_in: int, batch: int, k: int,
                     stream=None):
    _check("qdq_q8_0_logits_topk",
           lib().qdq_q8_0_logits_topk(_ptr(W), _ptr(x), _ptr(logits), _ptr(workspace), _ptr(index), _ptr(value),
                                      n_vocab, n_in, batch, k, _stream(stream)))


def gemm_batch_workspace_bytes(M: int, n_out: int, n_in: int) -> int:
    """Workspace bytes of the tensor-core batch GEMMs on the current device (the bf16 copy of X)."""
    return int(lib().qdq_gemm_batch_workspace_bytes(M, n_out, n_in))


def q8_0_gemm_batch(W, X, Y, workspace, n_out: int, n_in: int, M: int, stream=None):
    _check("qdq_q8_0_gemm_batch", lib().qdq_q8_0_gemm_batch(_ptr(W), _ptr(X), _ptr(Y), _ptr(workspace), n_out,
                                                            n_in, M, _stream(stream)))


def q4k_gemm_batch(W, X, Y, workspace, n_out: int, n_in: int, M: int, stream=None):
    _check("qdq_q4k_gemm_batch", lib().qdq_q4k_gemm_batch(_ptr(W), _ptr(X), _ptr(Y), _ptr(workspace), n_out,
                                                          n_in, M, _stream(stream)))


def q4k_swiglu_batch_workspace_bytes(M: int, n_ff: int, n_embd: int) -> int:
    return int(lib().qdq_q4k_swiglu_batch_workspace_bytes(M, n_ff, n_embd))


def q4k_swiglu_batch(Wg, Wu, X, mid, workspace, n_ff: int, n_embd: int, M: int, stream=None):
    _check("qdq_q4k_swiglu_batch", lib().qdq_q4k_swiglu_batch(_ptr(Wg), _ptr(Wu), _ptr(X), _ptr(mid),
                                                              _ptr(workspace), n_ff, n_embd, M, _stream(stream)))


def noop(stream=None):
    """One empty kernel on the stream (for the launch round-trip measurement)."""
    _check("qdq_noop", lib().qdq_noop(_stream(stream)))


def pipeline_timeouts() -> int:
    return int(lib().qdq_pipeline_timeouts())


def set_option(key: int, value: int) -> int:
    r = int(lib().qdq_set_option(key, value))
    if r < 0:
        raise QdqError("qdq_set_option", r)
    return r


# ---------------------------------------------------------------- decode-step operators
# (the element type and the row strides come from the tensors, whose first dimension is the rows; a tensor
# with fewer rows or elements than the call reads or writes raises ValueError)

_types = {}  # torch dtype -> QDQ_TYPE_*; filled at the first use, when torch is there


def _type(t) -> int:
    if not _types:
        import torch
        _types.update({torch.float32: QDQ_TYPE_F32, torch.float16: QDQ_TYPE_F16, torch.bfloat16: QDQ_TYPE_BF16})
        _of["int32"], _of["float32"] = torch.int32, torch.float32
    v = _types.get(t.dtype)
    if v is None:
        raise TypeError("float32, float16 or bfloat16 expected, got %s" % t.dtype)
    return v


_of = {}
_fast = None       # the C marshalling (_fastcall.so), bound to _fast_lib's functions
_fast_lib = None   # None: not tried yet; False: every call goes through the Python code


def _bind_fast():
    """Bind the C marshalling to the loaded library, once.  Where it was not built, or for another interpreter, and
    where nothing can be launched, the Python code makes the calls."""
    global _fast, _fast_lib
    import importlib.util
    import torch
    path = os.path.join(_PKG, "_fastcall.so")
    if not torch.cuda.is_available() or not os.path.exists(path):
        _fast_lib = False
        return
    handle = lib()
    try:
        spec = importlib.util.spec_from_file_location("_fastcall", path)
        m = importlib.util.module_from_spec(spec)
        spec.loader.exec_module(m)
    except ImportError:
        _fast_lib = False
        return
    m.bind(*[ctypes.cast(getattr(handle, f), ctypes.c_void_p).value for f in (
        "qdq_rms_norm", "qdq_kv_append", "qdq_kv_read", "qdq_kv_attention", "qdq_token_logprobs")],
        torch.float32, torch.float16, torch.bfloat16, torch.int32)
    _fast = m  # before _fast_lib, which sends other threads' calls to it
    _fast_lib = handle


def _vec(name, t, kind, least=0):
    """Address of a contiguous int32 or float32 tensor of at least so many elements, None for None (call _type first)."""
    if t is None:
        return None
    if t.dtype is not _of[kind] or not t.is_contiguous():
        raise TypeError("%s: a contiguous %s tensor expected" % (name, kind))
    if t.numel() < least:
        raise ValueError("%s: %d elements expected, got %d" % (name, least, t.numel()))
    return _cuda(name, t)


def _bytes(name, t, least=0):
    """Address of a contiguous tensor of at least so many bytes, None for None."""
    if t is None:
        return None
    if not t.is_contiguous():
        raise ValueError("%s: a contiguous tensor expected" % name)
    if t.nbytes < least:
        raise ValueError("%s: %d bytes expected, got %d" % (name, least, t.nbytes))
    return _cuda(name, t)


def _cuda(name, t):
    """Address of a CUDA tensor, None for None."""
    if t is None:
        return None
    if not t.is_cuda:
        raise TypeError("%s: a CUDA tensor expected" % name)
    return t.data_ptr()


def _rows(name, t, width, dtype, least=0):
    """(address, row stride) of a tensor of at least ``least`` rows: the first dimension, the others hold ``width`` packed
    elements (one dimension: one row)."""
    if t is None:
        return None, 0
    if t.dtype is not dtype:
        raise TypeError("%s: %s expected, got %s" % (name, dtype, t.dtype))
    shape, st = t.shape, t.stride()
    if len(shape) == 1:
        shape, st = (1, *shape), (width, *st)
    w = 1
    for d in range(len(shape) - 1, 0, -1):
        if shape[d] != 1 and st[d] != w:
            raise ValueError("%s: the elements of a row must be packed" % name)
        w *= shape[d]
    if w != width:
        raise ValueError("%s: rows of %d elements expected, got shape %s" % (name, width, tuple(t.shape)))
    if shape[0] < least:
        raise ValueError("%s: %d rows expected, got %d" % (name, least, shape[0]))
    return _cuda(name, t), st[0] if shape[0] > 1 else width


def rms_norm(x, weight, out, rows: int, n: int, eps: float = 1e-5, residual=None, sum_out=None, q8_out=None, stream=None):
    """RMS norm of ``x + residual`` per row into ``out`` (x's type) and / or ``q8_out`` (a packed Q8_0 matrix).

    ``sum_out`` receives ``x + residual``; it may be ``residual`` or ``x`` itself, and ``out`` may be ``x``."""
    if _fast_lib is None:
        _bind_fast()
    if _lib is _fast_lib:  # the ordinary case; None: something is unusual, and the code below says what
        status = _fast.rms_norm(x, weight, out, rows, n, eps, residual, sum_out, q8_out, _stream(stream))
        if status == 0:
            return
        if status is not None:
            raise QdqError("qdq_rms_norm", status)
    ty, dt = _type(x), x.dtype
    xp, xs = _rows("x", x, n, dt, rows)
    rp, rs = _rows("residual", residual, n, dt, rows)
    sp, ss = _rows("sum_out", sum_out, n, dt, rows)
    op, os_ = _rows("out", out, n, dt, rows)
    status = lib().qdq_rms_norm(xp, rp, _vec("weight", weight, "float32", n), sp, op, _bytes("q8_out", q8_out, rows * (n // 32) * 34), ty,
                                rows, n, xs, rs, ss, os_, eps, _stream(stream))
    if status != QDQ_OK:
        raise QdqError("qdq_rms_norm", status)


def kv_page_bytes(page_tokens: int, n_kv: int, head_dim: int) -> int:
    return int(lib().qdq_kv_page_bytes(page_tokens, n_kv, head_dim))


def kv_pages(n_pages: int, page_tokens: int, n_kv: int, head_dim: int, device="cuda"):
    """A pool of cache pages, zeroed: a uint8 tensor ``n_pages x kv_page_bytes``."""
    import torch
    b = kv_page_bytes(page_tokens, n_kv, head_dim)
    if b == 0:
        raise QdqError("qdq_kv_page_bytes", QDQ_ERR_UNSUPPORTED)
    return torch.zeros(n_pages, b, dtype=torch.uint8, device=device)


def _pool(pages, page_table, page_tokens, n_kv, head_dim):
    """(address of the pool, its pages, address of the table, its rows, their width)."""
    rec = (2 * page_tokens * head_dim + page_tokens // 2 + 127) // 128 * 128  # a head's record
    n, rest = divmod(pages.nbytes, n_kv * rec or 1)
    if rest or not pages.is_contiguous():
        raise ValueError("pages is not a whole number of packed pages")
    seqs, width = page_table.shape
    return _cuda("pages", pages), n, _vec("page_table", page_table, "int32"), seqs, width


def kv_append(pages, page_table, kv_len, k, v, n_kv: int, head_dim: int, page_tokens: int, cu_new=None, max_new: int = 1,
              stream=None):
    """Quantise new tokens (rows of ``k`` and ``v``) into the cache: the last tokens of each sequence's ``kv_len``."""
    if _fast_lib is None:
        _bind_fast()
    if _lib is _fast_lib:  # the ordinary case; None: something is unusual, and the code below says what
        status = _fast.kv_append(pages, page_table, kv_len, k, v, n_kv, head_dim, page_tokens, cu_new, max_new, _stream(stream))
        if status == 0:
            return
        if status is not None:
            raise QdqError("qdq_kv_append", status)
    ty, w = _type(k), n_kv * head_dim
    pp, n, tp, seqs, width = _pool(pages, page_table, page_tokens, n_kv, head_dim)
    least = seqs if cu_new is None else 0  # else the device knows how many rows there are
    kp, ks = _rows("k", k, w, k.dtype, least)
    vp, vs = _rows("v", v, w, k.dtype, least)
    status = lib().qdq_kv_append(pp, n, page_tokens, n_kv, head_dim, tp, width, _vec("kv_len", kv_len, "int32", seqs),
                                 _vec("cu_new", cu_new, "int32", seqs + 1), seqs, max_new, kp, vp, ks, vs, ty, _stream(stream))
    if status != QDQ_OK:
        raise QdqError("qdq_kv_append", status)


def kv_read(pages, page_table, start, cu, k, v, n_kv: int, head_dim: int, page_tokens: int, max_tokens: int, stream=None):
    """Write the values of cached tokens (``cu[s+1] - cu[s]`` of sequence s from ``start[s]``) to rows of ``k`` and ``v``."""
    if _fast_lib is None:
        _bind_fast()
    if _lib is _fast_lib:  # the ordinary case; None: something is unusual, and the code below says what
        status = _fast.kv_read(pages, page_table, start, cu, k, v, n_kv, head_dim, page_tokens, max_tokens, _stream(stream))
        if status == 0:
            return
        if status is not None:
            raise QdqError("qdq_kv_read", status)
    ty, w = _type(k), n_kv * head_dim
    pp, n, tp, seqs, width = _pool(pages, page_table, page_tokens, n_kv, head_dim)
    kp, ks = _rows("k", k, w, k.dtype)
    vp, vs = _rows("v", v, w, k.dtype)
    status = lib().qdq_kv_read(pp, n, page_tokens, n_kv, head_dim, tp, width, _vec("start", start, "int32", seqs),
                               _vec("cu", cu, "int32", seqs + 1), seqs, max_tokens, kp, vp, ks, vs, ty, _stream(stream))
    if status != QDQ_OK:
        raise QdqError("qdq_kv_read", status)


def kv_attention_workspace_bytes(n_seqs: int, max_q: int, max_kv_len: int, n_heads: int, n_kv: int, head_dim: int) -> int:
    return int(lib().qdq_kv_attention_workspace_bytes(n_seqs, max_q, max_kv_len, n_heads, n_kv, head_dim))


def kv_attention_workspace(n_seqs: int, max_q: int, max_kv_len: int, n_heads: int, n_kv: int, head_dim: int, device="cuda"):
    """A zeroed workspace of :func:`kv_attention`; calls on one stream may share it, also with :func:`token_logprobs`."""
    import torch
    return torch.zeros(kv_attention_workspace_bytes(n_seqs, max_q, max_kv_len, n_heads, n_kv, head_dim), dtype=torch.uint8,
                       device=device)


def kv_attention(pages, page_table, kv_len, q, out, workspace, n_heads: int, n_kv: int, head_dim: int, page_tokens: int,
                 max_kv_len: int, cu_q=None, max_q: int = 1, scale: float | None = None, softcap: float = 0.0,
                 window: int = 0, slopes=None, lse=None, stream=None):
    """Attention of the rows of ``q`` over the cached tokens into ``out`` (``scale`` defaults to head_dim ** -0.5)."""
    if _fast_lib is None:
        _bind_fast()
    if _lib is _fast_lib:  # the ordinary case; None: something is unusual, and the code below says what
        status = _fast.kv_attention(pages, page_table, kv_len, q, out, workspace, n_heads, n_kv, head_dim, page_tokens,
                                    max_kv_len, cu_q, max_q, head_dim ** -0.5 if scale is None else scale, softcap, window,
                                    slopes, lse, _stream(stream))
        if status == 0:
            return
        if status is not None:
            raise QdqError("qdq_kv_attention", status)
    ty, w = _type(q), n_heads * head_dim
    pp, n, tp, seqs, width = _pool(pages, page_table, page_tokens, n_kv, head_dim)
    least = seqs if cu_q is None else 0  # else the device knows how many rows there are
    qp, qs = _rows("q", q, w, q.dtype, least)
    op, os_ = _rows("out", out, w, q.dtype, least)
    status = lib().qdq_kv_attention(
        pp, n, page_tokens, n_kv, head_dim, tp, width, _vec("kv_len", kv_len, "int32", seqs),
        _vec("cu_q", cu_q, "int32", seqs + 1), seqs, max_q, max_kv_len, n_heads, qp, qs, op, os_,
        _vec("lse", lse, "float32", least * n_heads), _vec("slopes", slopes, "float32", n_heads),
        head_dim ** -0.5 if scale is None else scale, softcap, window, ty, _bytes("workspace", workspace), workspace.nbytes,
        _stream(stream))
    if status != QDQ_OK:
        raise QdqError("qdq_kv_attention", status)


def token_logprobs_workspace_bytes(rows: int, n: int, k: int) -> int:
    return int(lib().qdq_token_logprobs_workspace_bytes(rows, n, k))


def token_logprobs_workspace(rows: int, n: int, k: int, device="cuda"):
    """A zeroed workspace of :func:`token_logprobs`; calls on one stream may share it, also with :func:`kv_attention`."""
    import torch
    return torch.zeros(token_logprobs_workspace_bytes(rows, n, k), dtype=torch.uint8, device=device)


def token_logprobs(logits, tokens, logprob, entropy, rows: int, n: int, workspace, k: int = 0, top_index=None,
                   top_logprob=None, stream=None):
    """Per row: the log probability of ``tokens[r]``, the entropy, and the k best (index, log probability) pairs."""
    if _fast_lib is None:
        _bind_fast()
    if _lib is _fast_lib:  # the ordinary case; None: something is unusual, and the code below says what
        status = _fast.token_logprobs(logits, tokens, logprob, entropy, rows, n, workspace, k, top_index, top_logprob,
                                      _stream(stream))
        if status == 0:
            return
        if status is not None:
            raise QdqError("qdq_token_logprobs", status)
    ty = _type(logits)
    xp, xs = _rows("logits", logits, n, logits.dtype, rows)
    status = lib().qdq_token_logprobs(
        xp, xs, ty, _vec("tokens", tokens, "int32", rows), rows, n, k, _vec("logprob", logprob, "float32", rows),
        _vec("entropy", entropy, "float32", rows), _vec("top_index", top_index, "int32", rows * k),
        _vec("top_logprob", top_logprob, "float32", rows * k), _bytes("workspace", workspace), workspace.nbytes, _stream(stream))
    if status != QDQ_OK:
        raise QdqError("qdq_token_logprobs", status)


# ---------------------------------------------------------------- upload helpers
# (device memory comes from torch; the repack itself runs in the CUDA kernels)

def upload_q8_0(ggml_bytes, n_out: int, n_in: int, device="cuda", stream=None):
    """Copy raw GGML Q8_0 bytes (numpy uint8 or torch) to the device and repack them; returns the packed tensor."""
    import torch
    raw = torch.as_tensor(ggml_bytes, dtype=torch.uint8).reshape(-1).to(device)
    packed = torch.empty(q8_0_packed_bytes(n_out, n_in), dtype=torch.uint8, device=device)
    q8_0_pack(raw, packed, n_out, n_in, stream)
    return packed


def upload_q6k(ggml_bytes, n_out: int, n_in: int, device="cuda", stream=None):
    """Copy raw GGML Q6_K bytes (numpy uint8 or torch) to the device and repack them; returns the packed tensor."""
    import torch
    raw = torch.as_tensor(ggml_bytes, dtype=torch.uint8).reshape(-1).to(device)
    packed = torch.empty(q6k_packed_bytes(n_out, n_in), dtype=torch.uint8, device=device)
    q6k_pack(raw, packed, n_out, n_in, stream)
    return packed


def upload_q4k(ggml_bytes, n_out: int, n_in: int, device="cuda", stream=None):
    """Copy raw GGML Q4_K bytes (numpy uint8 or torch) to the device and repack them; returns the packed tensor."""
    import torch
    raw = torch.as_tensor(ggml_bytes, dtype=torch.uint8).reshape(-1).to(device)
    packed = torch.empty(q4k_packed_bytes(n_out, n_in), dtype=torch.uint8, device=device)
    q4k_pack(raw, packed, n_out, n_in, stream)
    return packed
