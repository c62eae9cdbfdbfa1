"""The paged key-value cache (include/kvpop_paged.h): argument marshalling only, as in ``_binding``.

A cache row is (sequence b, KV head h); its slots lie in pages taken from a pool that all sequences share.
A prompt fills it (``paged_compact_kv``), each step of decoding writes the new token's K and V into it, over
the token of least accumulated attention weight once the row is full (``paged_append_kv``), and attends to
it (``paged_decode_attention``, which also accumulates the weights that the eviction ranks by)::

    cache = kv.PagedCache.allocate(batch, n_kv_heads, head_dim, capacity=4032)
    kv.paged_compact_kv(k, v, keep, cu_seqlens, cache, score=target)
    while decoding:
        kv.paged_append_kv(k_new, v_new, cache, window=256, sinks=4)
        out, lse = kv.paged_decode_attention(q, cache, accumulate=True)

Given their buffers the calls neither allocate nor synchronise, and everything that changes from step to step
lives on the device, so the loop's body can be captured in a CUDA graph and replayed.
"""
from __future__ import annotations

import array
import contextlib
import ctypes
import math
import operator
import os

from . import _binding as _b

PAGED_HEADER_PATH = os.path.join(os.path.dirname(_b.HEADER_PATH), "kvpop_paged.h")

BF16, E4M3 = 0, 1


class CacheStruct(ctypes.Structure):
    _fields_ = [("k_pages", ctypes.c_void_p), ("v_pages", ctypes.c_void_p),
                ("k_stride", ctypes.c_int64 * 3), ("v_stride", ctypes.c_int64 * 3),
                ("pos_pages", ctypes.c_void_p), ("weight_pages", ctypes.c_void_p),
                ("k_scale", ctypes.c_void_p), ("v_scale", ctypes.c_void_p),
                ("page_table", ctypes.c_void_p), ("count", ctypes.c_void_p), ("seen", ctypes.c_void_p),
                ("n_pages", ctypes.c_int32), ("page_size", ctypes.c_int32), ("max_pages", ctypes.c_int32),
                ("batch", ctypes.c_int32), ("n_kv_heads", ctypes.c_int32), ("head_dim", ctypes.c_int32),
                ("capacity", ctypes.c_int32), ("dtype", ctypes.c_int32)]


_P, _I32, _I64, _SIZE = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t
_CACHE = ctypes.POINTER(CacheStruct)
SIGS = {
    "kvpop_paged_compact_kv": (ctypes.c_int, [_P, _P, _P, _P, _P, _I32, _CACHE, _P, _P]),
    "kvpop_paged_append_kv": (ctypes.c_int, [_P, _P, _I64, _P, _CACHE, _I32, _I32, _P, _P, _P]),
    "kvpop_paged_decode_workspace_bytes": (_SIZE, [_CACHE, _I32, _I32]),
    "kvpop_paged_decode_attention": (ctypes.c_int, [_P, _I64, _I32, _CACHE, ctypes.c_float, _I32, _P, _P, _P, _SIZE, _P,
                                                    _P]),
}


def paged_lib() -> ctypes.CDLL:
    """libkvpop.so with the paged cache's signatures set (they are declared beside kvpop.h's)."""
    h = _b._handle or _b.lib()
    if not getattr(h, "paged_ready", False):
        for name, (res, args) in SIGS.items():
            fn = getattr(h, name)
            fn.restype = res
            fn.argtypes = args
        h.paged_ready = True
    return h


# A call's host side is a few microseconds, so it asks torch for plain numbers instead of objects.

def _raw_stream(stream, device: int) -> int:
    import torch
    if stream is None:
        return torch._C._cuda_getCurrentRawStream(device)
    return _b._stream_ptr(stream)


def _host_i32(values, name: str) -> array.array:
    """int32 offsets on the host, of a list, a numpy array or a tensor."""
    if hasattr(values, "tolist"):
        values = values.tolist()
    try:
        return array.array("i", values)
    except OverflowError:
        raise ValueError(f"{name}: value out of int32 range") from None


def _i32(value, name: str) -> int:
    """A whole number within int32: ctypes would take its low 32 bits of any other."""
    try:
        value = operator.index(value)
    except TypeError:
        raise TypeError(f"{name} must be a whole number, not {value!r}") from None
    if not -2**31 <= value < 2**31:
        raise ValueError(f"{name} ({value}) is out of int32 range")
    return value


def _check_given(t, shape, dtype, device: int, name: str):
    import torch
    if (not isinstance(t, torch.Tensor) or t.dtype != dtype or t.shape != shape or t.get_device() != device
            or not t.is_contiguous()):
        raise ValueError(f"{name} must be a contiguous {dtype} CUDA tensor of shape {tuple(shape)} on cuda:{device}")


def _on_stream(stream):
    """A context in which torch allocates for `stream` (a torch stream or a raw handle), so that a buffer made here
    for a launch there is not handed to other work before that launch is done."""
    import torch
    if stream is None:
        return contextlib.nullcontext()
    if not hasattr(stream, "cuda_stream"):
        stream = torch.cuda.ExternalStream(int(stream))
    return torch.cuda.stream(stream)


class PagedCache:
    """The tensors of a paged cache, checked once; the calls below read and update them in place.

    k_pages, v_pages   [n_pages, H_kv, page_size, d] bf16 or float8_e4m3fn; any strides that are multiples of
                       16 bytes with d contiguous (token-major pages: pass ``pool.permute(0, 2, 1, 3)``)
    page_table         int32 [B, max_pages], contiguous; entries beyond a row's slots are not looked at
    count              int32 [B, H_kv], slots in use; < 0 marks a row that takes no part
    capacity           slots a row may use (default max_pages * page_size)
    seen               int32 [B, H_kv], tokens the sequence has had (appending)
    pos, weight        int32 / fp32 [n_pages, H_kv, page_size] (appending; weight also for accumulate=True)
    k_scale, v_scale   fp32 [H_kv], e4m3 caches: the pages hold K / k_scale and V / v_scale
    The tensors may be written by the caller between calls (a page table that grows, say), but not replaced.
    """

    def __init__(self, k_pages, v_pages, page_table, count, capacity: int | None = None, seen=None, pos=None,
                 weight=None, k_scale=None, v_scale=None):
        import torch
        if not isinstance(k_pages, torch.Tensor) or k_pages.dim() != 4 or not k_pages.is_cuda:
            raise TypeError("k_pages must be a 4-D CUDA tensor [n_pages, H_kv, page_size, d]")
        if k_pages.dtype not in (torch.bfloat16, torch.float8_e4m3fn):
            raise TypeError(f"k_pages must be bf16 or float8_e4m3fn, not {k_pages.dtype}")
        N, H, P, d = k_pages.shape
        dev = k_pages.device
        if (not isinstance(v_pages, torch.Tensor) or v_pages.dtype != k_pages.dtype or v_pages.shape != k_pages.shape
                or v_pages.device != dev):
            raise ValueError(f"v_pages must be a {k_pages.dtype} tensor of shape {tuple(k_pages.shape)} on {dev}")
        for name, t in (("k_pages", k_pages), ("v_pages", v_pages)):
            if t.stride(3) != 1 or any(t.stride(i) == 0 and t.shape[i] > 1 for i in range(3)):
                raise ValueError(f"{name} must have a contiguous last dimension and no broadcast ones")
        if not isinstance(page_table, torch.Tensor) or page_table.dim() != 2:
            raise TypeError("page_table must be a 2-D int32 CUDA tensor [B, max_pages]")
        B, max_pages = page_table.shape
        _b._tensor(page_table, (B, max_pages), torch.int32, dev, "page_table")
        _b._tensor(count, (B, H), torch.int32, dev, "count")
        if seen is not None:
            _b._tensor(seen, (B, H), torch.int32, dev, "seen")
        for name, t, dtype in (("pos", pos, torch.int32), ("weight", weight, torch.float32)):
            if t is not None:
                _b._tensor(t, (N, H, P), dtype, dev, name)
        for name, t in (("k_scale", k_scale), ("v_scale", v_scale)):
            if t is not None:
                if k_pages.dtype != torch.float8_e4m3fn:
                    raise ValueError(f"{name} is for float8_e4m3fn pages only")
                _b._tensor(t, (H,), torch.float32, dev, name)
        self.k_pages, self.v_pages, self.page_table, self.count = k_pages, v_pages, page_table, count
        self.seen, self.pos, self.weight, self.k_scale, self.v_scale = seen, pos, weight, k_scale, v_scale
        self.capacity = max_pages * P if capacity is None else int(capacity)
        if not 1 <= self.capacity <= max_pages * P:
            raise ValueError(f"capacity {self.capacity} is not within 1 .. max_pages * page_size = {max_pages * P}")
        self.batch, self.n_kv_heads, self.page_size, self.head_dim = B, H, P, d
        self.device, self.device_index = dev, k_pages.get_device()
        ptr = lambda t: None if t is None else t.data_ptr()
        strides = lambda t: (ctypes.c_int64 * 3)(*(t.stride(i) if t.shape[i] > 1 else 0 for i in range(3)))
        self.struct = CacheStruct(
            k_pages.data_ptr(), v_pages.data_ptr(), strides(k_pages), strides(v_pages), ptr(pos), ptr(weight),
            ptr(k_scale), ptr(v_scale), page_table.data_ptr(), count.data_ptr(), ptr(seen), N, P, max_pages, B, H, d,
            self.capacity, E4M3 if k_pages.dtype == torch.float8_e4m3fn else BF16)

    @classmethod
    def allocate(cls, batch: int, n_kv_heads: int, head_dim: int, capacity: int, page_size: int = 64, dtype=None,
                 k_scale=None, v_scale=None, device=None) -> "PagedCache":
        """An empty cache with pages of its own for every sequence."""
        import torch
        dev = torch.device("cuda", torch.cuda.current_device()) if device is None else torch.device(device)
        max_pages = -(-capacity // page_size)
        shape = (batch * max_pages, n_kv_heads, page_size)
        dtype = torch.bfloat16 if dtype is None else dtype
        pool = lambda: torch.empty((*shape, head_dim), dtype=dtype, device=dev)
        rows = lambda: torch.zeros((batch, n_kv_heads), dtype=torch.int32, device=dev)
        table = torch.arange(batch * max_pages, dtype=torch.int32, device=dev).view(batch, max_pages)
        return cls(pool(), pool(), table, rows(), capacity=capacity, seen=rows(),
                   pos=torch.full(shape, -1, dtype=torch.int32, device=dev), weight=torch.zeros(shape, device=dev),
                   k_scale=k_scale, v_scale=v_scale)


def _rows_of(t, shape, device: int, name: str) -> int:
    """The stride in elements between the first dimension's items of t (bf16, contiguous behind it), which may be
    a slice of a wider tensor such as a fused projection's output."""
    import torch
    if (not isinstance(t, torch.Tensor) or t.dtype != torch.bfloat16 or t.shape != shape
            or t.get_device() != device):
        raise ValueError(f"{name} must be a bf16 CUDA tensor of shape {shape} on cuda:{device}")
    s0, s1, s2 = t.stride()
    if s2 != 1 or (shape[1] > 1 and s1 != shape[2]):
        raise ValueError(f"{name} must be contiguous behind its first dimension")
    return s0 if shape[0] > 1 else shape[1] * shape[2]


def _check_cache(cache) -> int:
    import torch
    if not isinstance(cache, PagedCache):
        raise TypeError("cache must be a PagedCache")
    dev = cache.device_index
    if torch._C._cuda_getDevice() != dev:
        _b._on_current_device(cache, "the cache")
    return dev


def paged_compact_kv(k, v, keep, cu_seqlens, cache: PagedCache, score=None, status=None, stream=None) -> PagedCache:
    """Fills the cache from a packed prompt: the positions with keep = 1 (keep [H_kv, T] uint8, or None for every
    position), in order, up to the capacity; weight = score [H_kv, T] (or 0).  Writes pos, weight, count and seen."""
    import torch
    dev = _check_cache(cache)
    cu = _host_i32(cu_seqlens, "cu_seqlens")
    H, d = cache.n_kv_heads, cache.head_dim
    if not isinstance(k, torch.Tensor) or k.dim() != 3:
        raise TypeError("k must be a 3-D bf16 CUDA tensor [T, H_kv, d]")
    T = k.shape[0]
    _check_given(k, (T, H, d), torch.bfloat16, dev, "k")
    _check_given(v, (T, H, d), torch.bfloat16, dev, "v")
    if len(cu) != cache.batch + 1:
        raise ValueError(f"cu_seqlens describes {len(cu) - 1} sequences, the cache has {cache.batch}")
    if keep is not None:
        _check_given(keep, (H, T), torch.uint8, dev, "keep")
    if score is not None:
        _check_given(score, (H, T), torch.float32, dev, "score")
    _b._check(paged_lib().kvpop_paged_compact_kv(
        k.data_ptr(), v.data_ptr(), None if keep is None else keep.data_ptr(),
        None if score is None else score.data_ptr(), cu.buffer_info()[0], T, cache.struct,
        None if status is None else _b._status_ptr(status, cache.device), _raw_stream(stream, dev)))
    return cache


def paged_append_kv(k_new, v_new, cache: PagedCache, window: int, sinks: int, cu_new=None, evicted=None, status=None,
                    stream=None):
    """Appends new tokens [T_new, H_kv, d] (one per sequence, or cu_new [B + 1] offsets on the host) to every
    sequence, over the slots of least accumulated weight where a row is full.  Returns evicted [T_new, H_kv] int32:
    the position each token displaced, -1 for a free slot, -2 if it was not stored."""
    import torch
    window, sinks = _i32(window, "window"), _i32(sinks, "sinks")
    dev = _check_cache(cache)
    B, H, d = cache.batch, cache.n_kv_heads, cache.head_dim
    if cu_new is None:
        T, cu = B, None
    else:
        cu = _host_i32(cu_new, "cu_new")
        if len(cu) != B + 1:
            raise ValueError(f"cu_new describes {len(cu) - 1} sequences, the cache has {B}")
        T = cu[-1]
    stride = _rows_of(k_new, (T, H, d), dev, "k_new")
    if _rows_of(v_new, (T, H, d), dev, "v_new") != stride:
        raise ValueError("k_new and v_new must have the same stride between tokens")
    if evicted is not None:
        _check_given(evicted, (T, H), torch.int32, dev, "evicted")
    elif stream is None:
        evicted = k_new.new_empty((T, H), dtype=torch.int32)
    else:
        with _on_stream(stream):
            evicted = torch.empty((T, H), dtype=torch.int32, device=cache.device)
    if T == 0:
        return evicted
    _b._check(paged_lib().kvpop_paged_append_kv(
        k_new.data_ptr(), v_new.data_ptr(), stride, None if cu is None else cu.buffer_info()[0], cache.struct, window,
        sinks, evicted.data_ptr(), None if status is None else _b._status_ptr(status, cache.device),
        _raw_stream(stream, dev)))
    return evicted


def paged_decode_workspace_bytes(cache: PagedCache, n_q_heads: int, accumulate: bool | None = None) -> int:
    """Device workspace of paged_decode_attention (accumulate: whether weights are, by default if the cache has any)."""
    n_q_heads = _i32(int(n_q_heads), "n_q_heads")
    accumulate = cache.weight is not None if accumulate is None else accumulate
    return int(paged_lib().kvpop_paged_decode_workspace_bytes(cache.struct, n_q_heads, 1 if accumulate else 0))


def paged_decode_attention(q, cache: PagedCache, scale: float | None = None, accumulate: bool = False, out=None,
                           lse=None, workspace=None, status=None, stream=None):
    """One decode step over the cache: (out [B, H_q, d] bf16, lse [B, H_q] fp32); accumulate=True also adds each
    slot's attention weight, summed over the query heads of its KV head, to cache.weight."""
    import torch
    dev = _check_cache(cache)
    if not isinstance(q, torch.Tensor) or q.dim() != 3:
        raise TypeError("q must be a 3-D bf16 CUDA tensor [B, H_q, d]")
    B, d = cache.batch, cache.head_dim
    Hq = q.shape[1]
    shape = (B, Hq, d)
    stride = _rows_of(q, shape, dev, "q")
    h = paged_lib()
    with contextlib.nullcontext() if stream is None or (out is not None and lse is not None and workspace is not None) \
            else _on_stream(stream):
        if out is None:
            out = torch.empty(shape, dtype=torch.bfloat16, device=cache.device)
        else:
            _check_given(out, shape, torch.bfloat16, dev, "out")
        if lse is None:
            lse = torch.empty((B, Hq), dtype=torch.float32, device=cache.device)
        else:
            _check_given(lse, (B, Hq), torch.float32, dev, "lse")
        if workspace is None:
            need = h.kvpop_paged_decode_workspace_bytes(cache.struct, Hq, 1 if accumulate else 0)
            workspace = torch.empty(max(int(need), 256), dtype=torch.uint8, device=cache.device)
        elif (not isinstance(workspace, torch.Tensor) or workspace.get_device() != dev or not workspace.is_contiguous()):
            raise ValueError(f"workspace must be a contiguous CUDA tensor on cuda:{dev}")
    _b._check(h.kvpop_paged_decode_attention(
        q.data_ptr(), stride, Hq, cache.struct, 1.0 / math.sqrt(d) if scale is None else scale, 1 if accumulate else 0,
        out.data_ptr(), lse.data_ptr(), workspace.data_ptr(), workspace.nbytes,
        None if status is None else _b._status_ptr(status, cache.device), _raw_stream(stream, dev)))
    return out, lse
