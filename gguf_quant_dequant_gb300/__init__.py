"""Python binding of libqk (include/qk.h): argument marshalling only.

Every computation runs in the library's CUDA kernels; this module passes
device pointers, sizes and the current CUDA stream of PyTorch tensors, and
raises QKError on a non-zero status.  There is no CPU fallback: if libqk.so
has not been built, load() raises.  stream= of a call is a torch stream or a
raw handle; a result or a workspace that the call allocates for itself is then
taken as under torch.cuda.stream(stream).

Type ids: Q4_K = 1, Q6_K = 2, Q8_0 = 3, Q5_0 = 4, Q4_0 = 5, Q5_K = 6, Q2_K = 7, Q3_K = 8.
"""
from __future__ import annotations

import ctypes
import functools
import os
import threading

Q4_K, Q6_K, Q8_0, Q5_0, Q4_0, Q5_K, Q2_K, Q3_K = 1, 2, 3, 4, 5, 6, 7, 8
TYPES = {"Q4_K": Q4_K, "Q6_K": Q6_K, "Q8_0": Q8_0, "Q5_0": Q5_0, "Q4_0": Q4_0, "Q5_K": Q5_K, "Q2_K": Q2_K,
         "Q3_K": Q3_K}
OUT_F32, OUT_BF16 = 0, 1
STATUS = {0: "QK_OK", 1: "QK_ERR_TYPE", 2: "QK_ERR_SHAPE", 3: "QK_ERR_ALIGN", 4: "QK_ERR_NULL",
          5: "QK_ERR_WORKSPACE", 6: "QK_ERR_CUDA", 7: "QK_ERR_TIMEOUT", 8: "QK_ERR_ARG",
          9: "QK_ERR_FORMAT", 10: "QK_ERR_IO"}

LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libqk.so")
_lib = None
_lock = threading.Lock()

_p = ctypes.c_void_p
_i64 = ctypes.c_int64
_sz = ctypes.c_size_t
_int = ctypes.c_int
_u32 = ctypes.c_uint32
_u64 = ctypes.c_uint64
_f64p = ctypes.POINTER(ctypes.c_double)
_i64p = ctypes.POINTER(ctypes.c_int64)
_u64p = ctypes.POINTER(ctypes.c_uint64)


class GGUFTensorInfo(ctypes.Structure):
    """qk_gguf_tensor_info."""
    _fields_ = [("name", ctypes.c_char_p), ("n_dims", ctypes.c_uint32), ("dims", ctypes.c_int64 * 4),
                ("ggml_type", ctypes.c_uint32), ("qk_type", ctypes.c_int), ("offset", ctypes.c_uint64),
                ("nbytes", ctypes.c_uint64), ("data", ctypes.c_void_p)]


# name: (restype, argtypes), exactly as declared in include/qk.h
SIGNATURES = {
    "qk_version": (_int, []),
    "qk_block_bytes": (_sz, [_int]),
    "qk_block_elems": (_int, [_int]),
    "qk_row_bytes": (_sz, [_int, _i64]),
    "qk_dequant": (_int, [_int, _p, _i64, _i64, _p, _int, _p]),
    "qk_quantize": (_int, [_int, _p, _i64, _i64, _p, _p]),
    "qk_quantize_imatrix": (_int, [_int, _p, _i64, _i64, _p, _p, _p]),
    "qk_attn_decode_workspace": (ctypes.c_size_t, [_int, _i64, _int, _int, _int]),
    "qk_attn_decode": (_int, [_int, _p, _p, _p, _i64, _int, _int, _int, ctypes.c_float, _p, _p, ctypes.c_size_t, _p]),
    "qk_gemv_workspace": (_sz, [_int, _i64, _i64, _i64]),
    "qk_gemv": (_int, [_int, _p, _i64, _i64, _p, _i64, _p, _p, _sz, _p]),
    "qk_gemv_noalloc": (_int, [_int, _p, _i64, _i64, _p, _i64, _p, _p]),
    "qk_gemv_batch": (_int, [_int, _int, ctypes.POINTER(_p), ctypes.POINTER(_i64), _i64, _p,
                             ctypes.POINTER(_p), _p]),
    "qk_gemv_swiglu": (_int, [_int, _p, _p, _i64, _i64, _p, _p, _p]),
    "qk_gemm_workspace": (_sz, [_int, _i64, _i64, _i64]),
    "qk_gemm": (_int, [_int, _p, _i64, _i64, _p, _i64, _p, _p, _sz, _p]),
    "qk_kv_page_bytes": (_sz, [_int, _int, _int, _int]),
    "qk_kv_plan": (_int, [_p, _p, _p, _i64, _int, _p, _i64, _p, _i64, _p, _p, _p, _p, _p, _p, _p, _i64, _p]),
    "qk_kv_append": (_int, [_int, _p, _p, _int, _i64, _i64, _i64, _int, _int, _p, _p, _p, _i64, _int, _p]),
    "qk_kv_compact": (_int, [_int, _p, _p, _i64, _int, _int, _int, _p, _i64, _p, _p, _i64, _p, _i64, _p]),
    "qk_attn_tree_workspace": (_sz, [_int, _i64, _int, _i64, _int, _int, _int]),
    "qk_attn_tree": (_int, [_int, _p, _i64, _i64, _p, _p, _i64, _int, _p, _i64, _p, _p, _p, _i64, _int, _int, _int, _int,
                            ctypes.c_float, _p, _i64, _p, _sz, _p]),
    "qk_test_attn_tree_stalled": (_int, [_u32, _u32, _int, _p, _i64, _i64, _p, _p, _i64, _int, _p, _i64, _p, _p, _p, _i64,
                                         _int, _int, _int, _int, ctypes.c_float, _p, _i64, _p, _sz, _p]),
    "qk_logits_process": (_int, [_p, _int, _i64, _i64, _i64, _p, _i64, _p, _i64, _p, _p, _p, _p, _p, _p, _p, _p, _i64,
                                 _p, _p, _i64, _p, _i64, _p]),
    "qk_norm_rope": (_int, [_p, _p, _int, _i64, _i64, _i64, _int, _int, _int, _p, _p, _p, ctypes.c_float, _p, _int, _int, _p, _p,
                            _int, _i64, _i64, _p]),
    "qk_kv_append_rope": (_int, [_int, _p, _p, _p, _int, _i64, _i64, _i64, _i64, _int, _int, _int, _p, _p, _p, ctypes.c_float,
                                 _p, _int, _int, _p, _p, _p, _i64, _int, _p, _i64, _p]),
    "qk_verify_workspace": (_sz, [_i64, _i64, _i64]),
    "qk_verify_tree": (_int, [_p, _int, _i64, _i64, _i64, _p, _i64, _p, _p, _p, _p, _p, _p, _i64, _p, _i64, _p, _p, _p, _sz, _p]),
    "qk_moe_workspace": (_sz, [_int, _int, _int, _i64, _i64, _int, _i64]),
    "qk_moe_ffn": (_int, [_int, _p, _p, _int, _p, _int, _i64, _i64, _p, _int, _int, ctypes.c_float, _p, _i64, _p, _p, _p, _p,
                          _sz, _p]),
    "qk_test_moe_group": (_int, [_int, _int, _int, _i64, _i64, _int, _i64, _int, _int]),
    "qk_unpack": (_int, [_int, _p, _i64, _p, _p, _p, _p, _p, _p]),
    "qk_device_status": (_int, [_p]),
    "qk_test_stalled_wait": (_int, [ctypes.c_uint32, _p]),
    "qk_last_error": (ctypes.c_char_p, []),
    "qk_gguf_open": (_int, [ctypes.c_char_p, ctypes.POINTER(_p)]),
    "qk_gguf_parse": (_int, [_p, _u64, ctypes.POINTER(_p)]),
    "qk_gguf_close": (None, [_p]),
    "qk_gguf_version": (_u32, [_p]),
    "qk_gguf_n_kv": (_i64, [_p]),
    "qk_gguf_n_tensors": (_i64, [_p]),
    "qk_gguf_alignment": (_u64, [_p]),
    "qk_gguf_data_offset": (_u64, [_p]),
    "qk_gguf_image": (_p, [_p]),
    "qk_gguf_find_kv": (_i64, [_p, ctypes.c_char_p]),
    "qk_gguf_kv_key": (ctypes.c_char_p, [_p, _i64]),
    "qk_gguf_kv_type": (_int, [_p, _i64]),
    "qk_gguf_kv_int": (_int, [_p, _i64, _i64p]),
    "qk_gguf_kv_float": (_int, [_p, _i64, _f64p]),
    "qk_gguf_kv_str": (_p, [_p, _i64, _u64p]),
    "qk_gguf_kv_array": (_int, [_p, _i64, ctypes.POINTER(_int), _u64p]),
    "qk_gguf_kv_array_int": (_int, [_p, _i64, _u64, _i64p]),
    "qk_gguf_kv_array_float": (_int, [_p, _i64, _u64, _f64p]),
    "qk_gguf_kv_array_str": (_p, [_p, _i64, _u64, _u64p]),
    "qk_gguf_find_tensor": (_i64, [_p, ctypes.c_char_p]),
    "qk_gguf_tensor": (_int, [_p, _i64, ctypes.POINTER(GGUFTensorInfo)]),
}


class QKError(RuntimeError):
    def __init__(self, status: int, where: str, msg: str):
        super().__init__(f"{where}: {STATUS.get(status, status)}: {msg}")
        self.status = status


def load() -> ctypes.CDLL:
    """Load libqk.so (built in-tree by build.build()); raise if it is missing."""
    global _lib
    if _lib is not None:
        return _lib
    with _lock:
        if _lib is None:
            if not os.path.exists(LIB_PATH):
                raise RuntimeError(f"{LIB_PATH} is missing: build it with "
                                   "`python -m gguf_quant_dequant_gb300.build`")
            L = ctypes.CDLL(LIB_PATH)
            for name, (res, args) in SIGNATURES.items():
                fn = getattr(L, name)
                fn.restype = res
                fn.argtypes = args
            _lib = L
    return _lib


def _check(st: int, where: str) -> None:
    if st != 0:
        raise QKError(st, where, load().qk_last_error().decode())


def _stream(stream) -> int:
    import torch
    if stream is None:
        stream = torch.cuda.current_stream()
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def _stream_on(x, stream) -> int:
    """The current stream of x's device, or the given one."""
    if stream is not None:
        return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)
    import torch
    return torch._C._cuda_getCurrentRawStream(x.device.index)


def _empty(size, dtype, like, stream, kept: bool = True):
    """A new tensor beside `like` for a call on `stream`.  For another stream
    than the current one it comes from that stream's memory, as inside
    torch.cuda.stream(stream): the caching allocator could otherwise hand out
    bytes that earlier work of the current stream still uses, or hand them on
    while the call's kernels run.  kept: the caller gets the tensor and may use
    it on the current stream too."""
    import torch
    if stream is None or not like.is_cuda:
        return torch.empty(size, dtype=dtype, device=like.device)
    dev = like.device
    handle = _stream(stream)
    if handle == torch._C._cuda_getCurrentRawStream(dev.index):
        return torch.empty(size, dtype=dtype, device=dev)
    if not isinstance(stream, torch.cuda.Stream):
        stream = torch.cuda.ExternalStream(handle, dev) if handle else torch.cuda.default_stream(dev)
    with torch.cuda.stream(stream):
        x = torch.empty(size, dtype=dtype, device=dev)
    if kept:
        x.record_stream(torch.cuda.current_stream(dev))
    return x


def _ptr(t) -> int | None:
    return None if t is None else t.data_ptr()


def block_bytes(t: int) -> int:
    return load().qk_block_bytes(t)


def block_elems(t: int) -> int:
    return load().qk_block_elems(t)


def row_bytes(t: int, cols: int) -> int:
    return load().qk_row_bytes(t, cols)


def dequant(t: int, W, rows: int, cols: int, out=None, bf16: bool = False, stream=None):
    """W: uint8 CUDA tensor of packed blocks -> out [rows, cols] fp32 / bf16."""
    import torch
    if out is None:
        out = _empty((rows, cols), torch.bfloat16 if bf16 else torch.float32, W, stream)
    _check(load().qk_dequant(t, _ptr(W), rows, cols, _ptr(out), OUT_BF16 if bf16 else OUT_F32,
                             _stream(stream)), "qk_dequant")
    return out


def quantize(t: int, w, out=None, stream=None):
    """w: fp32 CUDA tensor [rows, cols] -> out: uint8 packed blocks, rows *
    row_bytes(t, cols) bytes (allocated when not given)."""
    import torch
    rows, cols = w.shape
    if out is None:
        out = _empty(rows * row_bytes(t, cols), torch.uint8, w, stream)
    _check(load().qk_quantize(t, _ptr(w), rows, cols, _ptr(out), _stream(stream)), "qk_quantize")
    return out


def quantize_imatrix(t: int, w, imp, out=None, stream=None):
    """w: fp32 CUDA [rows, cols], imp: fp32 CUDA [cols] column importances
    (mean squared activations) -> packed blocks minimising the
    importance-weighted error (qk_quantize_imatrix)."""
    import torch
    rows, cols = w.shape
    if out is None:
        out = _empty(rows * row_bytes(t, cols), torch.uint8, w, stream)
    _check(load().qk_quantize_imatrix(t, _ptr(w), rows, cols, _ptr(imp), _ptr(out), _stream(stream)),
           "qk_quantize_imatrix")
    return out


def attn_decode_workspace(t: int, T: int, n_heads: int, n_kv: int, d: int) -> int:
    return load().qk_attn_decode_workspace(t, T, n_heads, n_kv, d)


def attn_decode(t: int, q, K, V, T: int, n_heads: int, n_kv: int, d: int, scale: float, out=None, ws=None,
                stream=None):
    """Decode attention over a block-quantized KV cache (qk_attn_decode):
    q fp32 CUDA [n_heads, d]; K, V packed caches [T, n_kv, d] -> out fp32
    [n_heads, d]."""
    import torch
    if out is None:
        out = _empty((n_heads, d), torch.float32, q, stream)
    need = attn_decode_workspace(t, T, n_heads, n_kv, d)
    if ws is None:
        ws = _empty(max(need, 16), torch.uint8, q, stream, kept=False)
    _check(load().qk_attn_decode(t, _ptr(q), _ptr(K), _ptr(V), T, n_heads, n_kv, d, scale, _ptr(out), _ptr(ws),
                                 ws.numel() * ws.element_size(), _stream(stream)), "qk_attn_decode")
    return out


def gemv_swiglu(t: int, Wg, Wu, rows: int, cols: int, x, h=None, stream=None):
    """Decode SwiGLU: x fp32 CUDA [cols] -> h = SiLU(Wg x) * (Wu x), fp32 [rows]."""
    import torch
    if h is None:
        h = _empty(rows, torch.float32, x, stream)
    _check(load().qk_gemv_swiglu(t, _ptr(Wg), _ptr(Wu), rows, cols, _ptr(x), _ptr(h), _stream(stream)),
           "qk_gemv_swiglu")
    return h


def gemv_workspace(t: int, rows: int, cols: int, M: int) -> int:
    return load().qk_gemv_workspace(t, rows, cols, M)


def gemv(t: int, W, rows: int, cols: int, x, y=None, ws=None, stream=None):
    """x fp32 CUDA [M, cols] -> y fp32 [M, rows]; ws allocated if needed."""
    import torch
    M = x.shape[0] if x.dim() == 2 else 1
    if y is None:
        y = _empty((M, rows), torch.float32, x, stream)
    need = gemv_workspace(t, rows, cols, M)
    if ws is None and need:
        ws = _empty(need, torch.uint8, x, stream, kept=False)
    nbytes = 0 if ws is None else ws.numel() * ws.element_size()
    _check(load().qk_gemv(t, _ptr(W), rows, cols, _ptr(x), M, _ptr(y), _ptr(ws), nbytes, _stream(stream)),
           "qk_gemv")
    return y


def gemv_noalloc(t: int, W, rows: int, cols: int, x, y=None, stream=None):
    """qk_gemv_noalloc: qk_gemv for callers that cannot allocate device
    memory (no workspace; the GEMV needs none)."""
    import torch
    M = x.shape[0] if x.dim() == 2 else 1
    if y is None:
        y = _empty((M, rows), torch.float32, x, stream)
    _check(load().qk_gemv_noalloc(t, _ptr(W), rows, cols, _ptr(x), M, _ptr(y), _stream(stream)),
           "qk_gemv_noalloc")
    return y


def gemv_batch(t: int, Ws, rows, cols: int, x, ys=None, stream=None):
    """qk_gemv_batch: y_i = W_i x for matrices sharing one fp32 activation row
    x [cols] (or [1, cols]); returns the list of fp32 outputs [rows_i]."""
    import torch
    n = len(Ws)
    if ys is None:
        ys = [_empty(r, torch.float32, x, stream) for r in rows]
    Wp = (_p * n)(*[_ptr(w) for w in Ws])
    rp = (_i64 * n)(*rows)
    yp = (_p * n)(*[_ptr(y) for y in ys])
    _check(load().qk_gemv_batch(t, n, Wp, rp, cols, _ptr(x), yp, _stream(stream)), "qk_gemv_batch")
    return ys


def gemm_workspace(t: int, rows: int, cols: int, M: int) -> int:
    return load().qk_gemm_workspace(t, rows, cols, M)


def gemm(t: int, W, rows: int, cols: int, X, Y=None, ws=None, stream=None):
    """X bf16 CUDA [M, cols] -> Y fp32 [M, rows]."""
    import torch
    M = X.shape[0]
    if Y is None:
        Y = _empty((M, rows), torch.float32, X, stream)
    need = gemm_workspace(t, rows, cols, M)
    if ws is None and need:
        ws = _empty(need, torch.uint8, X, stream, kept=False)
    nbytes = 0 if ws is None else ws.numel() * ws.element_size()
    _check(load().qk_gemm(t, _ptr(W), rows, cols, _ptr(X), M, _ptr(Y), _ptr(ws), nbytes, _stream(stream)),
           "qk_gemm")
    return Y


# ------------------------------------- paged KV cache, tree attention, logits --
# These calls are a few microseconds on the GPU, so their checks are kept to
# what the C side cannot see: types, contiguity, element counts and that the
# memory is the GPU's.

TREE_MAX = 64


def _dtype(x, what: str) -> int:
    name = x.dtype.__str__()
    if name == "torch.float32":
        return OUT_F32
    if name == "torch.bfloat16":
        return OUT_BF16
    raise QKError(8, what, f"dtype {name}: float32 or bfloat16 expected")


def _on_gpu(x, what: str) -> None:
    if not x.is_cuda:
        raise QKError(8, what, f"a CUDA tensor expected, got one on {x.device}")


def _rows(x, what: str) -> int:
    """Elements from row to row of a CUDA tensor whose rows are contiguous."""
    shape, strides = x.shape, x.stride()
    want = 1
    for i in range(len(shape) - 1, 0, -1):
        if strides[i] != want and shape[i] != 1:
            raise QKError(8, what, f"strides {strides} of shape {tuple(shape)}: contiguous rows expected")
        want *= shape[i]
    if not x.is_cuda:
        _on_gpu(x, what)
    return strides[0] if shape[0] > 1 else want


def _of(x, dtype, what: str, n: int):
    """Pointer of a contiguous CUDA array of n elements of the type the C call
    reads; None for None."""
    if x is None:
        return None
    if x.dtype is not dtype or not x.is_contiguous():
        raise QKError(8, what, f"contiguous {dtype} expected, got {x.dtype} with strides {x.stride()}")
    if x.numel() != n:
        raise QKError(2, what, f"{n} elements expected, got shape {tuple(x.shape)}")
    if not x.is_cuda:
        _on_gpu(x, what)
    return x.data_ptr()


@functools.lru_cache(maxsize=256)
def kv_page_bytes(t: int, n_kv: int, d: int, page: int) -> int:
    return load().qk_kv_page_bytes(t, n_kv, d, page)


def _pool_pages(t: int, K, V, n_kv: int, d: int, page: int, what: str) -> int:
    import torch
    pb = kv_page_bytes(t, n_kv, d, page)
    if pb == 0:
        raise QKError(2, what, f"no paged cache of type {t} with n_kv={n_kv}, d={d}, page={page}")
    n = K.numel()
    if n % pb:
        raise QKError(2, what, f"K and V must be uint8 pools of the same whole number of {pb}-byte pages")
    _of(K, torch.uint8, what, n)
    _of(V, torch.uint8, what, n)
    return n // pb


def kv_plan(have, start, want, table, free_pages, n_free, page: int, cap: int, out=None, stream=None) -> dict:
    """Page bookkeeping of a step (qk_kv_plan): int32 CUDA have, start, want
    [n_req], table [n_req, P] and free_pages [F] (both updated in place), n_free
    [1] -> {"n_free" [1], "granted" [n_req], "cu" [n_req + 1], "slots" int64,
    "pos", "req" [cap]}.  out: a dict of such tensors to be written instead of
    new ones."""
    import torch
    n, P, F = have.shape[0], table.shape[1], free_pages.shape[0]
    i32, w = torch.int32, "kv_plan"
    ptrs = [_of(have, i32, w, n), _of(start, i32, w, n), _of(want, i32, w, n), _of(table, i32, w, n * P),
            _of(free_pages, i32, w, F), _of(n_free, i32, w, 1)]
    if out is None:
        e = _empty(2 + 2 * n + 2 * cap, i32, have, stream)
        slots = _empty(cap, torch.int64, have, stream)
        at, q = e.data_ptr(), slots.data_ptr()
        outs = (at, at + 4, at + 4 + 4 * n, q, at + 8 + 8 * n, at + 8 + 8 * n + 4 * cap)
        a, b, c, d, f = e.split((1, n, n + 1, cap, cap))
        out = {"n_free": a, "granted": b, "cu": c, "slots": slots, "pos": d, "req": f}
    else:
        outs = (_of(out["n_free"], i32, w, 1), _of(out["granted"], i32, w, n), _of(out["cu"], i32, w, n + 1),
                _of(out["slots"], torch.int64, w, cap), _of(out["pos"], i32, w, cap), _of(out["req"], i32, w, cap))
    _check(load().qk_kv_plan(ptrs[0], ptrs[1], ptrs[2], n, page, ptrs[3], P, ptrs[4], F, ptrs[5], outs[0], outs[1],
                             outs[2], outs[3], outs[4], outs[5], cap, _stream_on(have, stream)), "qk_kv_plan")
    return out


def kv_append(t: int, k, v, slots, K, V, page: int, stream=None) -> None:
    """Quantize k, v (fp32 or bf16 CUDA [n_tok, n_kv, d], rows contiguous) into
    the uint8 pools K, V at slots int64 [n_tok] (qk_kv_append)."""
    import torch
    n, n_kv, d = k.shape
    w = "kv_append"
    if v.shape != k.shape or v.dtype is not k.dtype:
        raise QKError(2, w, "k and v differ in shape or type")
    pages = _pool_pages(t, K, V, n_kv, d, page, w)
    _check(load().qk_kv_append(t, k.data_ptr(), v.data_ptr(), _dtype(k, w), n, _rows(k, w), _rows(v, w), n_kv, d,
                               _of(slots, torch.int64, w, n), K.data_ptr(), V.data_ptr(), pages, page,
                               _stream_on(k, stream)), "qk_kv_append")


def kv_compact(t: int, K, V, page: int, n_kv: int, d: int, table, base, path, n_path, stream=None) -> None:
    """Move the accepted rows base + path[:, j] to base + j (qk_kv_compact):
    int32 CUDA table [n_req, P], base, n_path [n_req], path [n_req, m]."""
    import torch
    w, i32, n, P, m = "kv_compact", torch.int32, base.shape[0], table.shape[1], path.shape[1]
    pages = _pool_pages(t, K, V, n_kv, d, page, w)
    _check(load().qk_kv_compact(t, K.data_ptr(), V.data_ptr(), pages, page, n_kv, d, _of(table, i32, w, n * P), P,
                                _of(base, i32, w, n), _of(path, i32, w, n * m), m, _of(n_path, i32, w, n), n,
                                _stream_on(K, stream)), "qk_kv_compact")


def _like_rows(out, n: int, h: int, d: int, dtype, like, stream, what: str):
    """out, or a new tensor, and its elements from row to row."""
    if out is None:
        return _empty((n, h, d), dtype, like, stream), h * d
    if out.dtype is not dtype or out.shape != (n, h, d):
        raise QKError(2, what, f"{dtype} of shape {(n, h, d)} expected, got {out.dtype} of {tuple(out.shape)}")
    return out, _rows(out, what)


def norm_rope(q, k, pos, freq, q_norm=None, k_norm=None, eps: float = 1e-6, pairs: bool = False, out_dtype=None, q_out=None,
              k_out=None, stream=None):
    """Norms of q and k heads and their rotation by position (qk_norm_rope): q
    [n_tok, n_heads, d], k [n_tok, n_kv, d] fp32 or bf16 CUDA (rows
    contiguous); pos int32 [n_tok], freq fp32 [rot / 2] (None: no rotation);
    q_norm, k_norm fp32 [d] or None -> (q_out, k_out) of out_dtype (q's own by
    default).  q or k may be None."""
    import torch
    w, f32 = "norm_rope", torch.float32
    x = q if q is not None else k
    if x is None:
        raise QKError(4, w, "q or k expected")
    n, _, d = x.shape
    hq, hk = 0 if q is None else q.shape[1], 0 if k is None else k.shape[1]
    if q is not None and k is not None and (k.dtype is not q.dtype or k.shape[0] != n or k.shape[2] != d):
        raise QKError(2, w, "q and k differ in type, tokens or width")
    out_dtype = out_dtype or x.dtype
    qs = ks = 0
    if q is not None:
        q_out, qs = _like_rows(q_out, n, hq, d, out_dtype, x, stream, w)
    if k is not None:
        k_out, ks = _like_rows(k_out, n, hk, d, out_dtype, x, stream, w)
    y = q_out if q is not None else k_out
    rot = 0 if freq is None else 2 * freq.shape[0]
    _check(load().qk_norm_rope(
        _ptr(q), _ptr(k), _dtype(x, w), n, 0 if q is None else _rows(q, w), 0 if k is None else _rows(k, w), hq, hk, d,
        _of(pos, torch.int32, w, n) if rot else None, _of(q_norm, f32, w, d), _of(k_norm, f32, w, d), eps, _of(freq, f32, w, rot // 2),
        rot, pairs, None if q is None else q_out.data_ptr(), None if k is None else k_out.data_ptr(), _dtype(y, w),
        qs, ks, _stream_on(x, stream)), "qk_norm_rope")
    return (q_out if q is not None else None), (k_out if k is not None else None)


def kv_append_rope(t: int, q, k, v, pos, freq, slots, K, V, page: int, q_norm=None, k_norm=None, eps: float = 1e-6,
                   pairs: bool = False, q_out=None, stream=None):
    """norm_rope on the way into the paged cache (qk_kv_append_rope): k, v
    [n_tok, n_kv, d] quantized into the uint8 pools K, V at slots int64 [n_tok],
    keys normed and rotated; q [n_tok, n_heads, d] (or None) -> q_out bf16."""
    import torch
    w, f32 = "kv_append_rope", torch.float32
    n, n_kv, d = k.shape
    if v.shape != k.shape or v.dtype is not k.dtype:
        raise QKError(2, w, "k and v differ in shape or type")
    h = qs = 0
    if q is not None:
        h = q.shape[1]
        if q.dtype is not k.dtype or q.shape[0] != n or q.shape[2] != d:
            raise QKError(2, w, "q and k differ in type, tokens or width")
        q_out, qs = _like_rows(q_out, n, h, d, torch.bfloat16, k, stream, w)
    pages = _pool_pages(t, K, V, n_kv, d, page, w)
    rot = 0 if freq is None else 2 * freq.shape[0]
    _check(load().qk_kv_append_rope(
        t, _ptr(q), k.data_ptr(), v.data_ptr(), _dtype(k, w), n, _rows(q, w) if h else 0, _rows(k, w), _rows(v, w), h, n_kv, d,
        _of(pos, torch.int32, w, n) if rot else None, _of(q_norm, f32, w, d), _of(k_norm, f32, w, d), eps, _of(freq, f32, w, rot // 2),
        rot, pairs, _of(slots, torch.int64, w, n), K.data_ptr(), V.data_ptr(), pages, page, q_out.data_ptr() if h else None,
        qs if h else 0, _stream_on(k, stream)), "qk_kv_append_rope")
    return q_out if q is not None else None


def attn_tree_workspace(t: int, n_req: int, max_q: int, max_pos: int, n_heads: int, n_kv: int, d: int) -> int:
    return load().qk_attn_tree_workspace(t, n_req, max_q, max_pos, n_heads, n_kv, d)


def attn_tree(t: int, q, K, V, page: int, n_kv: int, table, ctx, cu, mask, max_q: int, scale: float, out=None, ws=None,
              stream=None):
    """Attention of drafted-token trees over the paged cache (qk_attn_tree):
    q bf16 CUDA [n_tok, n_heads, d] (rows contiguous); table int32 [n_req, P],
    ctx int32 [n_req], cu int32 [n_req + 1], mask int64 [n_tok] (64 bits) or
    None -> out bf16 [n_tok, n_heads, d]."""
    return _attn_tree("qk_attn_tree", (), t, q, K, V, page, n_kv, table, ctx, cu, mask, max_q, scale, out, ws, stream)


def test_attn_tree_stalled(limit_us: int, tile: int, t: int, q, K, V, page: int, n_kv: int, table, ctx, cu, mask, max_q: int,
                           scale: float, out=None, ws=None, stream=None):
    """qk_test_attn_tree_stalled: attn_tree whose copies of V stop before each
    CTA's tile number `tile`, the wait for them limited to limit_us."""
    return _attn_tree("qk_test_attn_tree_stalled", (limit_us, tile), t, q, K, V, page, n_kv, table, ctx, cu, mask, max_q,
                      scale, out, ws, stream)


def _attn_tree(name: str, first: tuple, t, q, K, V, page, n_kv, table, ctx, cu, mask, max_q, scale, out, ws, stream):
    import torch
    w, i32 = "attn_tree", torch.int32
    n, n_heads, d = q.shape
    r, P = ctx.shape[0], table.shape[1]
    if q.dtype is not torch.bfloat16:
        raise QKError(8, w, "q must be bfloat16")
    if out is None:
        out = _empty((n, n_heads, d), torch.bfloat16, q, stream)
    elif out.dtype is not torch.bfloat16 or out.shape != q.shape:
        raise QKError(2, w, "out must be bfloat16 of q's shape")
    pages = _pool_pages(t, K, V, n_kv, d, page, w)
    L = load()
    if ws is None:
        ws = _empty(max(L.qk_attn_tree_workspace(t, r, max_q, P * page, n_heads, n_kv, d), 16), torch.uint8, q, stream,
                    kept=False)
    elif not (ws.is_cuda and ws.is_contiguous()):
        _on_gpu(ws, w)
        raise QKError(8, w, f"contiguous ws expected, got strides {ws.stride()}")
    _check(getattr(L, name)(*first, t, q.data_ptr(), n, _rows(q, w), K.data_ptr(), V.data_ptr(), pages, page,
                            _of(table, i32, w, r * P), P, _of(ctx, i32, w, r), _of(cu, i32, w, r + 1),
                            _of(mask, torch.int64, w, n), r, max_q, n_heads, n_kv, d, scale, out.data_ptr(), _rows(out, w),
                            ws.data_ptr(), ws.numel() * ws.element_size(), _stream_on(q, stream)), name)
    return out


def logits_process(logits, cu, hist, hist_len, rep, pres, freq, draft=None, mask=None, bias_tok=None, bias_val=None,
                   bias_len=None, grammar=None, out=None, stream=None):
    """Penalties, biases and grammar masks on logits (qk_logits_process):
    logits fp32 or bf16 CUDA [n_rows, vocab]; cu int32 [n_req + 1]; hist int32
    [n_req, H], hist_len int32, rep, pres, freq fp32 [n_req]; draft int32,
    mask int64 [n_rows]; bias_tok int32, bias_val fp32 [n_req, B], bias_len
    int32 [n_req]; grammar int32 [n_rows, words] -> out (may be logits)."""
    import torch
    w, i32, f32 = "logits_process", torch.int32, torch.float32
    n, V = logits.shape
    r, H = cu.shape[0] - 1, hist.shape[1]
    B = 0 if bias_tok is None else bias_tok.shape[1]
    words = 0 if grammar is None else grammar.shape[1]
    if out is None:
        out = _empty((n, V), logits.dtype, logits, stream)
    elif out.dtype is not logits.dtype or out.shape != logits.shape:
        raise QKError(2, w, "out must have the logits' type and shape")
    _check(load().qk_logits_process(
        logits.data_ptr(), _dtype(logits, w), n, V, _rows(logits, w), _of(cu, i32, w, r + 1), r, _of(hist, i32, w, r * H),
        H, _of(hist_len, i32, w, r), _of(rep, f32, w, r), _of(pres, f32, w, r), _of(freq, f32, w, r),
        _of(draft, i32, w, n), _of(mask, torch.int64, w, n), _of(bias_tok, i32, w, r * B),
        _of(bias_val, f32, w, r * B) if B else None, B, _of(bias_len, i32, w, r) if B else None,
        _of(grammar, i32, w, n * words), words, out.data_ptr(), _rows(out, w), _stream_on(logits, stream)),
        "qk_logits_process")
    return out


def moe_workspace(t: int, t_down: int, n_exp: int, rows: int, cols: int, k: int, n_tok: int) -> int:
    """Bytes for the current device (they follow from its number of SMs)."""
    return load().qk_moe_workspace(t, t_down, n_exp, rows, cols, k, n_tok)


_moe_need: dict = {}   # workspaces by device and sizes, of calls that went through


@functools.lru_cache(maxsize=256)
def _moe_bytes(t: int, t_down: int, n_exp: int, rows: int, cols: int) -> tuple:
    """Bytes of Wg (or Wu) and of Wd; (0, 0) where there is no such layer."""
    a, b = row_bytes(t, cols), row_bytes(t_down, rows)
    return (n_exp * rows * a, n_exp * cols * b) if a and b and n_exp > 0 else (0, 0)


def moe_ffn(t: int, Wg, Wu, t_down: int, Wd, n_exp: int, rows: int, cols: int, x, k: int, router=None, norm: bool = True,
            scale: float = 1.0, ids=None, gate=None, out=None, ws=None, stream=None):
    """A mixture-of-experts layer (qk_moe_ffn): packed uint8 Wg, Wu [n_exp,
    rows, cols] of type t, Wd [n_exp, cols, rows] of type t_down; x fp32 CUDA
    [n_tok, cols]; router fp32 [n_exp, cols], or None with ids int32 and gate
    fp32 [n_tok, k] given -> (out fp32 [n_tok, cols], ids, gate)."""
    import torch
    w, i32, f32 = "moe_ffn", torch.int32, torch.float32
    n = x.shape[0]
    up, down = _moe_bytes(t, t_down, n_exp, rows, cols)
    if not (up and down):
        raise QKError(2, w, f"no packed experts of n_exp={n_exp}, rows={rows}, cols={cols} in types {t}, {t_down}")
    if router is None and (ids is None or gate is None):
        raise QKError(4, w, "a router, or ids and gate, expected")
    if ids is None:
        ids = _empty((n, k), i32, x, stream)
    if gate is None:
        gate = _empty((n, k), f32, x, stream)
    if out is None:
        out = _empty((n, cols), f32, x, stream)
    sizes = need = None
    if ws is None:
        sizes = (x.device.index, t, t_down, n_exp, rows, cols, k, n)
        need = _moe_need.get(sizes) or moe_workspace(*sizes[1:])
        ws = _empty(max(need, 16), torch.uint8, x, stream, kept=False)
    elif not (ws.is_cuda and ws.is_contiguous()):
        _on_gpu(ws, w)
        raise QKError(8, w, f"contiguous ws expected, got strides {ws.stride()}")
    u8 = torch.uint8
    _check(load().qk_moe_ffn(t, _of(Wg, u8, w, up), _of(Wu, u8, w, up), t_down, _of(Wd, u8, w, down), n_exp, rows, cols,
                             _of(router, f32, w, n_exp * cols), k, norm, scale, _of(x, f32, w, n * cols), n, _of(ids, i32, w, n * k),
                             _of(gate, f32, w, n * k), _of(out, f32, w, n * cols), ws.data_ptr(), ws.numel() * ws.element_size(),
                             _stream_on(x, stream)), "qk_moe_ffn")
    if sizes is not None and sizes not in _moe_need:
        if len(_moe_need) >= 256:
            _moe_need.clear()
        _moe_need[sizes] = need
    return out, ids, gate


@functools.lru_cache(maxsize=256)
def verify_workspace(n_rows: int, n_req: int, vocab: int) -> int:
    return load().qk_verify_workspace(n_rows, n_req, vocab)


def verify_tree(logits, cu, draft, mask, temp, u_accept, u_sample, probs=None, max_path: int = TREE_MAX, out=None,
                ws=None, stream=None) -> dict:
    """Drafted trees judged against the target's probabilities (qk_verify_tree):
    logits fp32 or bf16 CUDA [n_rows, vocab]; cu int32 [n_req + 1]; draft
    int32, mask int64 (or None: chains), u_accept fp32 [n_rows]; temp, u_sample
    fp32 [n_req]; probs fp32 [n_rows, vocab] or None -> {"path", "tokens" int32
    [n_req, max_path], "n_path" int32 [n_req]}.  out: such a dict to be written
    instead of new tensors."""
    import torch
    w, i32, f32 = "verify_tree", torch.int32, torch.float32
    n, V = logits.shape
    r = cu.shape[0] - 1
    if probs is not None and (probs.dtype is not f32 or probs.shape != logits.shape):
        raise QKError(2, w, "probs must be float32 of the logits' shape")
    if out is None:
        shape = (r, max_path)   # three tensors: views of one cost the host more
        out = {"path": _empty(shape, i32, logits, stream), "tokens": _empty(shape, i32, logits, stream),
               "n_path": _empty(r, i32, logits, stream)}
    elif out["path"].dim() != 2:
        raise QKError(2, w, f"path of two dimensions expected, got shape {tuple(out['path'].shape)}")
    P = out["path"].shape[1]
    need = verify_workspace(n, r, V)
    if ws is None and need:
        ws = _empty(need, torch.uint8, logits, stream, kept=False)
    elif ws is not None and not (ws.is_cuda and ws.is_contiguous()):
        _on_gpu(ws, w)
        raise QKError(8, w, f"contiguous ws expected, got strides {ws.stride()}")
    _check(load().qk_verify_tree(
        logits.data_ptr(), _dtype(logits, w), n, V, _rows(logits, w), _of(cu, i32, w, r + 1), r, _of(draft, i32, w, n),
        _of(mask, torch.int64, w, n), _of(temp, f32, w, r), _of(u_accept, f32, w, n), _of(u_sample, f32, w, r), _ptr(probs),
        0 if probs is None else _rows(probs, w), _of(out["path"], i32, w, r * P), P, _of(out["n_path"], i32, w, r),
        _of(out["tokens"], i32, w, r * P), _ptr(ws), 0 if ws is None else ws.numel() * ws.element_size(), _stream_on(logits, stream)),
        "qk_verify_tree")
    return out


def unpack(t: int, W, nblocks: int, stream=None):
    """-> (codes int16 [nblocks, elems], sc int16 [nblocks, 16], mins uint8
    [nblocks, 16], d f32 [nblocks], dmin f32 [nblocks]) as CUDA tensors."""
    import torch
    codes = _empty((nblocks, block_elems(t)), torch.int16, W, stream)
    sc = _empty((nblocks, 16), torch.int16, W, stream)
    mins = _empty((nblocks, 16), torch.uint8, W, stream)
    d = _empty(nblocks, torch.float32, W, stream)
    dmin = _empty(nblocks, torch.float32, W, stream)
    _check(load().qk_unpack(t, _ptr(W), nblocks, _ptr(codes), _ptr(sc), _ptr(mins), _ptr(d), _ptr(dmin),
                            _stream(stream)), "qk_unpack")
    return codes, sc, mins, d, dmin


def test_stalled_wait(limit_us: int, stream=None) -> None:
    """qk_test_stalled_wait: a bounded wait on a barrier nothing arrives on."""
    _check(load().qk_test_stalled_wait(limit_us, _stream(stream)), "qk_test_stalled_wait")


def device_status(stream=None) -> None:
    _check(load().qk_device_status(_stream(stream)), "qk_device_status")


# ------------------------------------------------------------ GGUF reader --

_V_STR, _V_ARR, _V_F32, _V_F64 = 8, 9, 6, 12


class GGUF:
    """A parsed GGUF image (qk_gguf_*): header, metadata and tensor infos.
    Open a file (memory-mapped) with GGUF(path=...) or parse bytes the object
    keeps alive with GGUF(data=...).  Tensor data stays in the image."""

    def __init__(self, path: str | None = None, data: bytes | None = None):
        L = load()
        h = _p()
        self._buf = None
        if path is not None:
            _check(L.qk_gguf_open(os.fsencode(path), ctypes.byref(h)), "qk_gguf_open")
        else:
            self._buf = ctypes.create_string_buffer(bytes(data), len(data))
            _check(L.qk_gguf_parse(ctypes.cast(self._buf, _p), len(data), ctypes.byref(h)), "qk_gguf_parse")
        self._h = h

    def close(self) -> None:
        if self._h:
            load().qk_gguf_close(self._h)
            self._h = _p()

    def __enter__(self):
        return self

    def __exit__(self, *exc):
        self.close()

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    @property
    def version(self) -> int:
        return load().qk_gguf_version(self._h)

    @property
    def alignment(self) -> int:
        return load().qk_gguf_alignment(self._h)

    @property
    def data_offset(self) -> int:
        return load().qk_gguf_data_offset(self._h)

    def keys(self) -> list:
        L = load()
        return [L.qk_gguf_kv_key(self._h, i).decode() for i in range(L.qk_gguf_n_kv(self._h))]

    def kv_type(self, key: str) -> int:
        L = load()
        return L.qk_gguf_kv_type(self._h, L.qk_gguf_find_kv(self._h, key.encode()))

    def _str(self, ptr, n) -> str:
        return ctypes.string_at(ptr, n.value).decode("utf-8", "surrogateescape") if n.value else ""

    def kv(self, key: str):
        """The value of `key` as int / float / str / list (KeyError if absent)."""
        L = load()
        i = L.qk_gguf_find_kv(self._h, key.encode())
        if i < 0:
            raise KeyError(key)
        t = L.qk_gguf_kv_type(self._h, i)
        n = ctypes.c_uint64()
        if t == _V_STR:
            return self._str(L.qk_gguf_kv_str(self._h, i, ctypes.byref(n)), n)
        if t in (_V_F32, _V_F64):
            v = ctypes.c_double()
            _check(L.qk_gguf_kv_float(self._h, i, ctypes.byref(v)), "qk_gguf_kv_float")
            return v.value
        if t == _V_ARR:
            et = _int()
            _check(L.qk_gguf_kv_array(self._h, i, ctypes.byref(et), ctypes.byref(n)), "qk_gguf_kv_array")
            out = []
            for j in range(n.value):
                if et.value == _V_STR:
                    m = ctypes.c_uint64()
                    out.append(self._str(L.qk_gguf_kv_array_str(self._h, i, j, ctypes.byref(m)), m))
                elif et.value in (_V_F32, _V_F64):
                    v = ctypes.c_double()
                    _check(L.qk_gguf_kv_array_float(self._h, i, j, ctypes.byref(v)), "qk_gguf_kv_array_float")
                    out.append(v.value)
                elif et.value == _V_ARR:
                    raise QKError(1, "GGUF.kv", "nested arrays are not exposed")
                else:
                    v = ctypes.c_int64()
                    _check(L.qk_gguf_kv_array_int(self._h, i, j, ctypes.byref(v)), "qk_gguf_kv_array_int")
                    out.append(v.value)
            return out
        v = ctypes.c_int64()
        _check(L.qk_gguf_kv_int(self._h, i, ctypes.byref(v)), "qk_gguf_kv_int")
        return v.value

    def tensors(self) -> list:
        L = load()
        return [self._info(i) for i in range(L.qk_gguf_n_tensors(self._h))]

    def _info(self, i: int) -> dict:
        info = GGUFTensorInfo()
        _check(load().qk_gguf_tensor(self._h, i, ctypes.byref(info)), "qk_gguf_tensor")
        return {"name": info.name.decode(), "dims": list(info.dims[:info.n_dims]), "ggml_type": info.ggml_type,
                "qk_type": info.qk_type, "offset": info.offset, "nbytes": info.nbytes, "data": info.data}

    def tensor(self, name: str) -> dict:
        i = load().qk_gguf_find_tensor(self._h, name.encode())
        if i < 0:
            raise KeyError(name)
        return self._info(i)

    def tensor_bytes(self, name: str) -> bytes:
        """A copy of the tensor's data bytes."""
        t = self.tensor(name)
        return ctypes.string_at(t["data"], t["nbytes"])
