"""Python binding of libqgemv (ctypes, argument marshalling only).

Every entry point has the C name without the ``qgemv_`` prefix.  Tensors are passed as
raw device pointers (``tensor.data_ptr()``); PyTorch is used for device memory and
streams only.  All work runs in the CUDA library; if it is missing this module raises.
"""
from __future__ import annotations

import ctypes
import os

from .build import LIB

Q4_K, NVFP4, TQ1_0, Q5_K, Q6_K, Q8_0 = 0, 1, 2, 3, 4, 5
OPT_FORCE_PATH, OPT_RING_DEPTH, OPT_ROWS_PER_STAGE, OPT_SPIN_LIMIT_NS, OPT_PDL, OPT_TEST_STALL, OPT_CTAS_PER_SM, \
    OPT_KSPLIT, OPT_GRID_PER_SM = 0, 2, 3, 4, 5, 6, 7, 8, 9
STATUS = {0: "QGEMV_OK", 1: "QGEMV_ERR_INVALID_ARG", 2: "QGEMV_ERR_UNSUPPORTED_FORMAT", 3: "QGEMV_ERR_BAD_SHAPE",
          4: "QGEMV_ERR_MISALIGNED", 5: "QGEMV_ERR_CUDA", 6: "QGEMV_ERR_TIMEOUT", 7: "QGEMV_ERR_OOM",
          8: "QGEMV_ERR_NO_DEVICE", 9: "QGEMV_ERR_TOO_LARGE", 10: "QGEMV_ERR_BAD_INDEX"}
OK, ERR_INVALID_ARG, ERR_UNSUPPORTED_FORMAT, ERR_BAD_SHAPE, ERR_MISALIGNED, ERR_CUDA, ERR_TIMEOUT, ERR_OOM, \
    ERR_NO_DEVICE, ERR_TOO_LARGE, ERR_BAD_INDEX = range(11)
NOALLOC_MAX_COLUMN_SUMS = 262144  # QGEMV_NOALLOC_MAX_COLUMN_SUMS
OUT_F32, OUT_F16, OUT_BF16 = 0, 1, 2
KV_F16, KV_BF16, KV_E4M3 = 1, 2, 3
MAX_GROUP = 8  # QGEMV_MAX_GROUP
MAX_BATCH = 8  # QGEMV_MAX_BATCH


class Problem(ctypes.Structure):
    """qgemv_problem_t: one matrix of run_group."""
    _fields_ = [("fmt", ctypes.c_int), ("packed_W", ctypes.c_void_p), ("packed_W_up", ctypes.c_void_p),
                ("N", ctypes.c_int64), ("y", ctypes.c_void_p), ("alpha", ctypes.c_float),
                ("beta", ctypes.c_float), ("out", ctypes.c_int), ("swiglu", ctypes.c_int)]


class KvCache(ctypes.Structure):
    """qgemv_kv_cache_t: a paged key-value cache."""
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("k_scale", ctypes.c_void_p),
                ("v_scale", ctypes.c_void_p), ("page_stride", ctypes.c_int64), ("scale_stride", ctypes.c_int64),
                ("pages", ctypes.c_int32), ("page_size", ctypes.c_int32), ("kv_heads", ctypes.c_int32),
                ("head_dim", ctypes.c_int32), ("type", ctypes.c_int)]


class PagePlan(ctypes.Structure):
    """qgemv_page_plan_t: block tables and slot maps of one step."""
    _fields_ = [("cached", ctypes.c_void_p), ("fresh", ctypes.c_void_p), ("table", ctypes.c_void_p),
                ("table_stride", ctypes.c_int64), ("free_pages", ctypes.c_void_p), ("free_count", ctypes.c_void_p),
                ("lens", ctypes.c_void_p), ("offsets", ctypes.c_void_p), ("slots", ctypes.c_void_p),
                ("positions", ctypes.c_void_p), ("owners", ctypes.c_void_p), ("counts", ctypes.c_void_p),
                ("capacity", ctypes.c_int64), ("requests", ctypes.c_int32), ("table_width", ctypes.c_int32),
                ("page_size", ctypes.c_int32)]


class KvStore(ctypes.Structure):
    """qgemv_kv_store_t: q and k rotated, k and v stored in the cache."""
    _fields_ = [("cache", KvCache), ("q", ctypes.c_void_p), ("k", ctypes.c_void_p), ("v", ctypes.c_void_p),
                ("q_stride", ctypes.c_int64), ("k_stride", ctypes.c_int64), ("v_stride", ctypes.c_int64),
                ("q_out", ctypes.c_void_p), ("q_out_stride", ctypes.c_int64), ("slots", ctypes.c_void_p),
                ("positions", ctypes.c_void_p), ("rope", ctypes.c_void_p), ("tokens", ctypes.c_int64),
                ("rope_positions", ctypes.c_int32), ("rot_dim", ctypes.c_int32), ("interleaved", ctypes.c_int32),
                ("q_heads", ctypes.c_int32), ("in_type", ctypes.c_int), ("q_type", ctypes.c_int)]


class AttnDecode(ctypes.Structure):
    """qgemv_attn_decode_t: one new token per request over the paged cache."""
    _fields_ = [("cache", KvCache), ("q", ctypes.c_void_p), ("q_stride", ctypes.c_int64), ("out", ctypes.c_void_p),
                ("out_stride", ctypes.c_int64), ("lse", ctypes.c_void_p), ("table", ctypes.c_void_p),
                ("table_stride", ctypes.c_int64), ("lens", ctypes.c_void_p), ("scale", ctypes.c_float),
                ("window", ctypes.c_int32), ("requests", ctypes.c_int32), ("table_width", ctypes.c_int32),
                ("q_heads", ctypes.c_int32), ("type", ctypes.c_int)]


class Lora(ctypes.Structure):
    """qgemv_lora_t: low-rank adapters added to a projection's output."""
    _fields_ = [("x", ctypes.c_void_p), ("x_stride", ctypes.c_int64), ("A", ctypes.c_void_p), ("B", ctypes.c_void_p),
                ("ids", ctypes.c_void_p), ("ranks", ctypes.c_void_p), ("scales", ctypes.c_void_p),
                ("base", ctypes.c_void_p), ("y", ctypes.c_void_p), ("y_stride", ctypes.c_int64),
                ("rows", ctypes.c_int64), ("N", ctypes.c_int64), ("K", ctypes.c_int64), ("adapters", ctypes.c_int32),
                ("rank", ctypes.c_int32), ("type", ctypes.c_int), ("out", ctypes.c_int)]


EXPORTS = ["qgemv_create", "qgemv_destroy", "qgemv_run", "qgemv_unpack", "qgemv_check_error",
           "qgemv_status_string", "qgemv_packed_bytes", "qgemv_group_size", "qgemv_set_option",
           "qgemv_describe", "qgemv_build_marker", "qgemv_run_noalloc", "qgemv_run_group", "qgemv_run_ex", "qgemv_run_batch",
           "qgemv_run_gemm", "qgemv_page_plan", "qgemv_kv_store", "qgemv_attn_decode", "qgemv_run_lora"]

_lib = None


class QgemvError(RuntimeError):
    def __init__(self, status: int, where: str):
        super().__init__(f"{where}: {STATUS.get(status, status)} ({status_string(status)})")
        self.status = status


def lib() -> ctypes.CDLL:
    """Load the in-tree libqgemv.so (raises if it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB):
            raise ImportError(f"libqgemv.so is not built ({LIB}); run __graft_entry__.build()")
        L = ctypes.CDLL(LIB)
        vp, i64, st = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int
        L.qgemv_create.argtypes = [ctypes.POINTER(vp), ctypes.c_int]
        L.qgemv_destroy.argtypes = [vp]
        L.qgemv_run.argtypes = [vp, ctypes.c_int, vp, vp, i64, i64, vp, vp]
        L.qgemv_unpack.argtypes = [vp, ctypes.c_int, vp, i64, i64, vp, vp, vp, vp]
        L.qgemv_check_error.argtypes = [vp, vp]
        L.qgemv_status_string.argtypes = [ctypes.c_int]
        L.qgemv_status_string.restype = ctypes.c_char_p
        L.qgemv_packed_bytes.argtypes = [ctypes.c_int, i64, i64]
        L.qgemv_packed_bytes.restype = ctypes.c_size_t
        L.qgemv_group_size.argtypes = [ctypes.c_int]
        L.qgemv_set_option.argtypes = [vp, ctypes.c_int, i64]
        L.qgemv_describe.argtypes = [vp, ctypes.c_int, i64, i64, ctypes.c_char_p, ctypes.c_size_t]
        L.qgemv_build_marker.restype = ctypes.c_char_p
        L.qgemv_run_noalloc.argtypes = [ctypes.c_int, vp, vp, i64, i64, vp, vp]
        L.qgemv_run_group.argtypes = [vp, vp, i64, ctypes.c_int, ctypes.POINTER(Problem), vp]
        L.qgemv_run_ex.argtypes = [vp, ctypes.c_int, vp, vp, i64, i64, ctypes.c_float, ctypes.c_float, vp,
                                   ctypes.c_int, vp]
        L.qgemv_run_batch.argtypes = [vp, ctypes.c_int, vp, ctypes.c_int, vp, i64, i64, vp, vp]
        L.qgemv_run_gemm.argtypes = [vp, ctypes.c_int, vp, i64, vp, i64, i64, vp, vp]
        L.qgemv_page_plan.argtypes = [vp, ctypes.POINTER(PagePlan), vp]
        L.qgemv_kv_store.argtypes = [vp, ctypes.POINTER(KvStore), vp]
        L.qgemv_attn_decode.argtypes = [vp, ctypes.POINTER(AttnDecode), vp]
        L.qgemv_run_lora.argtypes = [vp, ctypes.POINTER(Lora), vp]
        for name in ("qgemv_create", "qgemv_destroy", "qgemv_run", "qgemv_unpack", "qgemv_check_error",
                     "qgemv_set_option", "qgemv_describe", "qgemv_run_noalloc", "qgemv_run_group",
                     "qgemv_run_ex", "qgemv_run_batch", "qgemv_run_gemm", "qgemv_page_plan", "qgemv_kv_store",
                     "qgemv_attn_decode", "qgemv_run_lora"):
            getattr(L, name).restype = st
        _lib = L
    return _lib


def _ptr(t) -> int | None:
    if t is None:
        return None
    if isinstance(t, int):
        return t
    return t.data_ptr()


def _first_current_stream() -> int:
    """The current stream's handle.  torch.cuda.current_stream() builds an object for it, 3 us a call, as long as a
    small launch takes in all; after the first call (which initialises CUDA) the plain handle is asked for."""
    global _current_stream
    import torch
    handle = torch.cuda.current_stream().cuda_stream
    raw, device = getattr(torch._C, "_cuda_getCurrentRawStream", None), getattr(torch._C, "_cuda_getDevice", None)
    if raw is not None and device is not None and raw(device()) == handle:
        _current_stream = lambda: raw(device())  # noqa: E731
    else:
        _current_stream = lambda: torch.cuda.current_stream().cuda_stream  # noqa: E731
    return handle


_current_stream = _first_current_stream


def _stream(stream) -> int | None:
    if stream is None:
        return _current_stream()
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _check(status: int, where: str) -> None:
    if status != OK:
        raise QgemvError(status, where)


def status_string(status: int) -> str:
    return lib().qgemv_status_string(status).decode()


def build_marker() -> str:
    return lib().qgemv_build_marker().decode()


def packed_bytes(fmt: int, N: int, K: int) -> int:
    return lib().qgemv_packed_bytes(fmt, N, K)


def group_size(fmt: int) -> int:
    return lib().qgemv_group_size(fmt)


class Handle:
    """Owns a qgemv_handle_t (split-K workspace and error word on one device)."""

    def __init__(self, device: int = 0):
        h = ctypes.c_void_p()
        _check(lib().qgemv_create(ctypes.byref(h), device), "qgemv_create")
        self._h = h
        self.device = device

    @property
    def ptr(self):
        return self._h

    def close(self) -> None:
        if self._h is not None and self._h.value:
            lib().qgemv_destroy(self._h)
        self._h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


def create(device: int = 0) -> Handle:
    return Handle(device)


def destroy(h: Handle) -> None:
    h.close()


def run(h: Handle, fmt: int, x, packed_W, N: int, K: int, y, stream=None, check: bool = True) -> int:
    """y = x . dequant(W)^T, asynchronous on `stream` (default: torch's current stream)."""
    st = lib().qgemv_run(h.ptr, fmt, _ptr(x), _ptr(packed_W), N, K, _ptr(y), _stream(stream))
    if check:
        _check(st, "qgemv_run")
    return st


def run_noalloc(fmt: int, x, packed_W, N: int, K: int, y, stream=None, check: bool = True) -> int:
    """qgemv_run_noalloc: the same GEMV without a handle, using the library's fixed scratch
    (for callers that may not allocate device memory).  Calls must not overlap on the GPU."""
    st = lib().qgemv_run_noalloc(fmt, _ptr(x), _ptr(packed_W), N, K, _ptr(y), _stream(stream))
    if check:
        _check(st, "qgemv_run_noalloc")
    return st


def run_ex(h: Handle, fmt: int, x, packed_W, N: int, K: int, y, alpha: float = 1.0, beta: float = 0.0,
           out: int = OUT_F32, stream=None, check: bool = True) -> int:
    """y = alpha * x . dequant(W)^T + beta * y, y of type `out` (OUT_F32 / OUT_F16 / OUT_BF16)."""
    st = lib().qgemv_run_ex(h.ptr, fmt, _ptr(x), _ptr(packed_W), N, K, alpha, beta, _ptr(y), out,
                            _stream(stream))
    if check:
        _check(st, "qgemv_run_ex")
    return st


def run_batch(h: Handle, fmt: int, x, M: int, packed_W, N: int, K: int, y, stream=None, check: bool = True) -> int:
    """Y[m] = X[m] . dequant(W)^T for M (<= MAX_BATCH) row-major activation vectors x [M, K]."""
    st = lib().qgemv_run_batch(h.ptr, fmt, _ptr(x), M, _ptr(packed_W), N, K, _ptr(y), _stream(stream))
    if check:
        _check(st, "qgemv_run_batch")
    return st


def run_gemm(h: Handle, fmt: int, x, M: int, packed_W, N: int, K: int, y, stream=None, check: bool = True) -> int:
    """Y = X . dequant(W)^T for any number M of row-major activation rows x [M, K] (NVFP4 with
    M > MAX_BATCH on the tcgen05 tensor-core kernel)."""
    st = lib().qgemv_run_gemm(h.ptr, fmt, _ptr(x), M, _ptr(packed_W), N, K, _ptr(y), _stream(stream))
    if check:
        _check(st, "qgemv_run_gemm")
    return st


def problem(fmt: int, packed_W, N: int, y, packed_W_up=None, alpha: float = 1.0, beta: float = 0.0,
            out: int = OUT_F32, swiglu: bool = False) -> Problem:
    return Problem(fmt, _ptr(packed_W), _ptr(packed_W_up), N, _ptr(y), alpha, beta, out, int(swiglu))


def run_group(h: Handle, x, K: int, problems, stream=None, check: bool = True) -> int:
    """GEMVs sharing x (a list of `problem(...)` entries, at most MAX_GROUP), one launch."""
    arr = (Problem * max(1, len(problems)))(*problems)
    st = lib().qgemv_run_group(h.ptr, _ptr(x), K, len(problems), arr, _stream(stream))
    if check:
        _check(st, "qgemv_run_group")
    return st


def unpack(h: Handle, fmt: int, packed_W, N: int, K: int, codes, scales, mins=None, stream=None,
           check: bool = True) -> int:
    st = lib().qgemv_unpack(h.ptr, fmt, _ptr(packed_W), N, K, _ptr(codes), _ptr(scales), _ptr(mins),
                            _stream(stream))
    if check:
        _check(st, "qgemv_unpack")
    return st


def check_error(h: Handle, stream=None) -> int:
    return lib().qgemv_check_error(h.ptr, _stream(stream))


def set_option(h: Handle, opt: int, value: int, check: bool = True) -> int:
    st = lib().qgemv_set_option(h.ptr, opt, value)
    if check:
        _check(st, "qgemv_set_option")
    return st


def describe(h: Handle, fmt: int, N: int, K: int) -> str:
    buf = ctypes.create_string_buffer(512)
    _check(lib().qgemv_describe(h.ptr, fmt, N, K, buf, 512), "qgemv_describe")
    return buf.value.decode()


# ------------------------------------------------------------------ serving a batch of requests
# The calls below are described by a struct that a program builds once and keeps while its
# buffers stay where they are.  The *_desc functions fill one from tensors (shapes and strides
# are taken from them) and hold on to the tensors; everything else is checked by the library.
def _elem(t, allowed, what) -> int:
    import torch
    types = {torch.float32: OUT_F32, torch.float16: OUT_F16, torch.bfloat16: OUT_BF16}
    if types.get(t.dtype) not in allowed:
        raise TypeError(f"{what}: unsupported element type {t.dtype}")
    return types[t.dtype]


def _want(t, dtype, what, ndim=None):
    """`t`, checked to be a contiguous device tensor of `dtype` (None stays None)."""
    if t is None:
        return None
    if not t.is_cuda or not t.is_contiguous() or t.dtype != dtype or (ndim is not None and t.dim() != ndim):
        raise TypeError(f"{what}: a contiguous {dtype} device tensor"
                        f"{'' if ndim is None else f' of {ndim} dimensions'} is wanted")
    return t


def _rows(t, what) -> int:
    """The row stride of a device tensor [rows, ...] whose rows are contiguous."""
    inner = 1
    for size, stride in zip(reversed(t.shape[1:]), reversed(t.stride()[1:])):
        if size != 1 and stride != inner:
            raise TypeError(f"{what}: the elements of a row have to be contiguous")
        inner *= size
    if not t.is_cuda:
        raise TypeError(f"{what}: a device tensor is wanted")
    return t.stride(0) if t.shape[0] > 1 else inner


def _size(t, n, what):
    if t is not None and t.numel() != n:
        raise ValueError(f"{what}: {n} elements are wanted, got {t.numel()}")


def _table(t, what):
    import torch
    if not t.is_cuda or t.dtype != torch.int32 or t.dim() != 2 or (t.shape[1] > 1 and t.stride(1) != 1):
        raise TypeError(f"{what}: an int32 device tensor [requests, pages] with contiguous rows is wanted")
    return t.stride(0) if t.shape[0] > 1 else t.shape[1]


def kv_cache(k, v, k_scale=None, v_scale=None) -> KvCache:
    """The cache in tensors k and v [pages, kv_heads, page_size, head_dim] (fp16, bf16, or e4m3 codes as uint8
    or float8_e4m3fn with fp32 scales [pages, kv_heads, page_size]); only the page stride is free."""
    import torch
    types = {torch.float16: KV_F16, torch.bfloat16: KV_BF16, torch.uint8: KV_E4M3, torch.float8_e4m3fn: KV_E4M3}
    if k.dtype not in types or v.dtype != k.dtype or k.dim() != 4 or k.shape != v.shape or k.stride() != v.stride():
        raise TypeError("kv_cache: k and v of one shape, layout and cache type are wanted")
    pages, heads, size, dim = k.shape
    stride = max(_rows(k, "kv_cache: k"), _rows(v, "kv_cache: v"))
    scale_stride = 0
    if types[k.dtype] == KV_E4M3:
        for t in (k_scale, v_scale):
            if t is None or t.dtype != torch.float32 or t.shape != k.shape[:3] or t.stride() != k_scale.stride():
                raise TypeError("kv_cache: an e4m3 cache has fp32 scales [pages, kv_heads, page_size]")
        scale_stride = max(_rows(k_scale, "kv_cache: k_scale"), _rows(v_scale, "kv_cache: v_scale"))
    c = KvCache(_ptr(k), _ptr(v), _ptr(k_scale), _ptr(v_scale), stride, scale_stride, pages, size, heads, dim,
                types[k.dtype])
    c.keep = (k, v, k_scale, v_scale)
    return c


def page_plan_desc(cached, fresh, table, free, free_count, page, lens, slots, counts, offsets=None, positions=None,
                   owners=None) -> PagePlan:
    """Plan of one step: requests with `cached` tokens bring `fresh` new ones; pages come from the top of the
    stack free[0 .. free_count).  The number of slots is the step's token capacity."""
    import torch
    i32, n, cap = torch.int32, cached.numel(), slots.numel()
    for t, what in ((cached, "cached"), (fresh, "fresh"), (free, "free"), (free_count, "free_count"), (lens, "lens"),
                    (counts, "counts"), (offsets, "offsets"), (positions, "positions"), (owners, "owners")):
        _want(t, i32, f"page_plan: {what}", 1)
    _want(slots, torch.int64, "page_plan: slots", 1)
    for t, size, what in ((fresh, n, "fresh"), (lens, n, "lens"), (offsets, n + 1, "offsets"), (counts, 4, "counts"),
                          (positions, cap, "positions"), (owners, cap, "owners"), (free_count, 1, "free_count")):
        _size(t, size, f"page_plan: {what}")
    stride = _table(table, "page_plan: table")
    if table.shape[0] != n:
        raise ValueError("page_plan: one row of the table per request is wanted")
    d = PagePlan(_ptr(cached), _ptr(fresh), _ptr(table), stride, _ptr(free), _ptr(free_count), _ptr(lens),
                 _ptr(offsets), _ptr(slots), _ptr(positions), _ptr(owners), _ptr(counts), cap, n, table.shape[1], page)
    d.keep = (cached, fresh, table, free, free_count, lens, offsets, slots, positions, owners, counts)
    return d


def page_plan(h: Handle, desc: PagePlan, stream=None, check: bool = True) -> int:
    """Fill the block table, lengths and slot map that `desc` (page_plan_desc) describes."""
    st = lib().qgemv_page_plan(h.ptr, desc, _stream(stream))
    if check:
        _check(st, "qgemv_page_plan")
    return st


def kv_store_desc(cache: KvCache, k, v, slots, positions, rope=None, interleaved: bool = False, q=None,
                  q_out=None) -> KvStore:
    """k and v [tokens, kv_heads * head_dim] (rows may be slices of wider ones) into `cache`, k and q rotated by
    rope [positions, rot_dim] (cosines, then sines); q [tokens, q_heads * head_dim] into q_out."""
    import torch
    tokens = k.shape[0]
    kinds = (OUT_F32, OUT_F16, OUT_BF16)
    _want(slots, torch.int64, "kv_store: slots", 1)
    _want(positions, torch.int32, "kv_store: positions", 1)
    _want(rope, torch.float32, "kv_store: rope", 2)
    _size(slots, tokens, "kv_store: slots")
    _size(positions, tokens, "kv_store: positions")
    width = cache.kv_heads * cache.head_dim
    for t, what in ((k, "k"), (v, "v")):
        if t.shape[0] != tokens or t.numel() != tokens * width:
            raise ValueError(f"kv_store: {what} [tokens, kv_heads * head_dim] is wanted")
    if v.dtype != k.dtype or (q is not None and q.dtype != k.dtype) or (q is None) != (q_out is None):
        raise TypeError("kv_store: q, k and v of one type, and q together with q_out, are wanted")
    heads, q_type, q_stride, qo_stride = 0, OUT_F16, 0, 0
    if q is not None:
        if tokens and q.numel() % (tokens * cache.head_dim) or q.shape[0] != tokens or q_out.shape[0] != tokens \
                or q_out.numel() != q.numel():
            raise ValueError("kv_store: q and q_out [tokens, q_heads * head_dim] are wanted")
        heads = q[:1].numel() // cache.head_dim if tokens else 1
        q_type = _elem(q_out, (OUT_F16, OUT_BF16), "kv_store: q_out")
        q_stride, qo_stride = _rows(q, "kv_store: q"), _rows(q_out, "kv_store: q_out")
    d = KvStore(cache, _ptr(q), _ptr(k), _ptr(v), q_stride, _rows(k, "kv_store: k"), _rows(v, "kv_store: v"),
                _ptr(q_out), qo_stride, _ptr(slots), _ptr(positions), _ptr(rope), tokens,
                0 if rope is None else rope.shape[0], 0 if rope is None else rope.shape[1], int(interleaved), heads,
                _elem(k, kinds, "kv_store: k"), q_type)
    d.keep = (getattr(cache, "keep", None), q, k, v, q_out, slots, positions, rope)
    return d


def kv_store(h: Handle, desc: KvStore, stream=None, check: bool = True) -> int:
    """Rotate and store the rows that `desc` (kv_store_desc) describes."""
    st = lib().qgemv_kv_store(h.ptr, desc, _stream(stream))
    if check:
        _check(st, "qgemv_kv_store")
    return st


def attn_decode_desc(cache: KvCache, q, table, lens, out, scale: float, window: int = 0, lse=None) -> AttnDecode:
    """One query row [q_heads, head_dim] per request over the first lens[r] tokens of its pages (the last
    `window` of them when that is not 0); out like q, lse fp32 [requests, q_heads]."""
    import torch
    n = q.shape[0]
    if q.dim() != 3 or q.shape[2] != cache.head_dim or out.shape != q.shape or out.dtype != q.dtype:
        raise ValueError("attn_decode: q and out [requests, q_heads, head_dim] of one type are wanted")
    _want(lens, torch.int32, "attn_decode: lens", 1)
    _want(lse, torch.float32, "attn_decode: lse", 2)
    _size(lens, n, "attn_decode: lens")
    _size(lse, n * q.shape[1], "attn_decode: lse")
    stride = _table(table, "attn_decode: table")
    if table.shape[0] != n:
        raise ValueError("attn_decode: one row of the table per request is wanted")
    d = AttnDecode(cache, _ptr(q), _rows(q, "attn_decode: q"), _ptr(out), _rows(out, "attn_decode: out"), _ptr(lse),
                   _ptr(table), stride, _ptr(lens), scale, window, n, table.shape[1], q.shape[1],
                   _elem(q, (OUT_F16, OUT_BF16), "attn_decode: q"))
    d.keep = (getattr(cache, "keep", None), q, out, lse, table, lens)
    return d


def attn_decode(h: Handle, desc: AttnDecode, stream=None, check: bool = True) -> int:
    """The attention that `desc` (attn_decode_desc) describes."""
    st = lib().qgemv_attn_decode(h.ptr, desc, _stream(stream))
    if check:
        _check(st, "qgemv_attn_decode")
    return st


def lora_desc(x, A, B, ids, y, base=None, ranks=None, scales=None) -> Lora:
    """y[m] = base[m] + scales[a] * B[a] (A[a] x[m]) with a = ids[m] (-1: none); x [rows, K],
    A [adapters, rank, K], B [adapters, N, rank], base and y [rows, N]."""
    import torch
    adapters, rank, K = A.shape
    rows, N = y.shape
    _want(A, x.dtype, "run_lora: A", 3)
    _want(B, x.dtype, "run_lora: B", 3)
    _want(ids, torch.int32, "run_lora: ids", 1)
    _want(ranks, torch.int32, "run_lora: ranks", 1)
    _want(scales, torch.float32, "run_lora: scales", 1)
    if x.shape != (rows, K) or B.shape != (adapters, N, rank):
        raise ValueError("run_lora: x [rows, K], A [adapters, rank, K] and B [adapters, N, rank] are wanted")
    _size(ids, rows, "run_lora: ids")
    _size(ranks, adapters, "run_lora: ranks")
    _size(scales, adapters, "run_lora: scales")
    y_stride = _rows(y, "run_lora: y")
    if base is not None and (base.shape != y.shape or base.dtype != y.dtype or _rows(base, "run_lora: base") != y_stride):
        raise ValueError("run_lora: base has to have y's shape, type and row stride")
    d = Lora(_ptr(x), _rows(x, "run_lora: x"), _ptr(A), _ptr(B), _ptr(ids), _ptr(ranks), _ptr(scales), _ptr(base),
             _ptr(y), y_stride, rows, N, K, adapters, rank, _elem(x, (OUT_F16, OUT_BF16), "run_lora: x"),
             _elem(y, (OUT_F32, OUT_F16, OUT_BF16), "run_lora: y"))
    d.keep = (x, A, B, ids, ranks, scales, base, y)
    return d


def run_lora(h: Handle, desc: Lora, stream=None, check: bool = True) -> int:
    """Add the adapters that `desc` (lora_desc) describes."""
    st = lib().qgemv_run_lora(h.ptr, desc, _stream(stream))
    if check:
        _check(st, "qgemv_run_lora")
    return st
