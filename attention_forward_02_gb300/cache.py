"""The 8-bit paged KV cache on torch tensors (include/fa.h, "The 8-bit paged KV cache").

    cache = FACache.empty(num_pages, heads, page, d)          # e4m3, or dtype=torch.int8
    fa_cache_write(cache, k, v, page_table, seq_lens)         # k, v [T, heads, d]
    seq_lens += T // B
    o, lse = fa_decode_cache(q, cache, page_table, seq_lens)  # q [B, Hq, Nq, d]

or, over the best pages of a long cache,

    pages = fa_cache_select(q, cache, page_table, seq_lens, slots)
    o, lse = fa_decode_cache(q, cache, page_table, seq_lens, pages=pages)

and ``k, v = fa_cache_read(cache, page_table, seq_lens, N)`` for ``fa_fwd`` or
``fa_decode``.  ``page_table`` [B, max_pages] and ``seq_lens`` [B] are int32 CUDA
tensors; the calls read them on the device, so a captured graph replays with
whatever they hold then.  What they hold cannot be checked by the call: a page
number or length outside the cache is left out, and
``fa_last_device_status`` reports it.
"""
from ctypes import byref
from typing import NamedTuple, Optional

import torch

from ._lib import (FA_BF16, FA_E4M3, FA_FP16, FA_INT8, CacheDesc, FAError, fa_cache_read_raw,
                   fa_cache_select_raw, fa_cache_select_workspace_size, fa_cache_write_raw,
                   fa_decode_cache_raw, fa_decode_cache_workspace_size)

_CODES = {torch.float16: FA_FP16, torch.bfloat16: FA_BF16}
_FORMATS = {torch.float8_e4m3fn: FA_E4M3, torch.int8: FA_INT8}


class FACache(NamedTuple):
    """The buffers of a cache: codes k, v [num_pages, heads, page, d] (float8_e4m3fn or int8), scales
    [num_pages, heads] fp32 and, for ``fa_cache_select``, the pages' mean keys k_mean int8
    [num_pages, heads, d] with their scales.  Nothing is kept beside them."""
    k: torch.Tensor
    v: torch.Tensor
    k_scale: torch.Tensor
    v_scale: torch.Tensor
    k_mean: Optional[torch.Tensor] = None
    k_mean_scale: Optional[torch.Tensor] = None

    @classmethod
    def empty(cls, num_pages, heads, page, d, dtype=torch.float8_e4m3fn, device="cuda", means=True):
        """A cache with nothing in it (its memory is not initialised).  means: with mean keys."""
        if dtype not in _FORMATS:
            raise FAError(2, "cache dtype must be float8_e4m3fn or int8, got %s" % dtype)
        k, v = (torch.empty((num_pages, heads, page, d), dtype=dtype, device=device) for _ in range(2))
        ks, vs, ms = (torch.empty((num_pages, heads), dtype=torch.float32, device=device)
                      for _ in range(3))
        if not means:
            return cls(k, v, ks, vs)
        mean = torch.empty((num_pages, heads, d), dtype=torch.int8, device=device)
        return cls(k, v, ks, vs, mean, ms)


def _describe(cache):
    """The checked CacheDesc of a cache."""
    if not isinstance(cache, FACache):
        raise FAError(1, "cache must be an FACache")
    k, v, ks, vs, mean, ms = cache
    if not isinstance(k, torch.Tensor) or k.dim() != 4 or k.dtype not in _FORMATS:
        raise FAError(1, "the cache's k must be [num_pages, heads, page, d] of float8_e4m3fn or int8")
    num_pages, heads, page, d = k.shape
    device, pair = k.device, (num_pages, heads)
    wanted = ((k, "k", k.shape, k.dtype), (v, "v", k.shape, k.dtype),
              (ks, "k_scale", pair, torch.float32), (vs, "v_scale", pair, torch.float32))
    if mean is not None or ms is not None:
        wanted += ((mean, "k_mean", (num_pages, heads, d), torch.int8),
                   (ms, "k_mean_scale", pair, torch.float32))
    for t, name, shape, dtype in wanted:
        if (not isinstance(t, torch.Tensor) or not t.is_cuda or t.device != device or t.shape != shape
                or t.dtype != dtype or not t.is_contiguous()):
            raise FAError(1, "the cache's %s must be a contiguous CUDA tensor %s of %s on %s"
                          % (name, tuple(shape), dtype, device))
    return CacheDesc(k.data_ptr(), v.data_ptr(), ks.data_ptr(), vs.data_ptr(),
                     mean.data_ptr() if mean is not None else None,
                     ms.data_ptr() if ms is not None else None, num_pages, heads, page, d,
                     _FORMATS[k.dtype])


def _check_batch(device, page_table, seq_lens):
    for t, name, dim in ((page_table, "page_table", 2), (seq_lens, "seq_lens", 1)):
        if (not isinstance(t, torch.Tensor) or t.device != device or t.dtype != torch.int32
                or t.dim() != dim or (t.numel() and t.stride(-1) != 1)):
            raise FAError(1, "%s must be a %d-dimensional int32 tensor on %s, its last dimension "
                          "contiguous" % (name, dim, device))
    B = seq_lens.shape[0]
    if page_table.shape[0] != B:
        raise FAError(1, "page_table and seq_lens must have one row for each sequence")
    P = page_table.shape[1]
    return B, page_table.stride(0) if B > 1 else P, P


def _code(t, name):
    code = _CODES.get(t.dtype)
    if code is None:
        raise FAError(2, "%s must be float16 or bfloat16, got %s" % (name, t.dtype))
    return code


def _strides(t):
    """Element strides of all dimensions but the last; those of a dimension of one do not matter."""
    return [s if n > 1 else 0 for s, n in zip(t.stride()[:-1], t.shape[:-1])]


def _rows(t, name, dim, device, heads, d):
    """Checks an input whose rows of d values are contiguous; returns its type's code."""
    if (not isinstance(t, torch.Tensor) or t.device != device or t.dim() != dim or t.shape[-1] != d
            or (t.numel() and t.stride(-1) != 1) or (heads is not None and t.shape[1] != heads)):
        raise FAError(1, "%s must be a %d-dimensional CUDA tensor of rows of %d contiguous values on "
                      "%s%s" % (name, dim, d, device, " with %d heads" % heads if heads else ""))
    return _code(t, name)


def _output(t, name, shape, dtype, device):
    if (not isinstance(t, torch.Tensor) or t.device != device or t.shape != shape or t.dtype != dtype
            or not t.is_contiguous()):
        raise FAError(1, "%s must be a contiguous CUDA tensor %s of %s on %s" % (name, shape, dtype, device))
    return t


class _On:
    """The device and stream of a call; memory that is allocated inside belongs to that stream."""

    def __init__(self, device, stream):
        if stream is not None and stream.device != device:
            raise FAError(1, "the stream must be one of %s" % device)
        self.stream = stream
        self.within = torch.cuda.device(device) if stream is None else torch.cuda.stream(stream)
        self.device = device

    def __enter__(self):
        self.within.__enter__()
        if self.stream is None:
            return torch.cuda.current_stream(self.device).cuda_stream
        return self.stream.cuda_stream

    def __exit__(self, *exc):
        return self.within.__exit__(*exc)


def _workspace(workspace, need, device):
    if workspace is None:
        return torch.empty(max(need, 16), dtype=torch.uint8, device=device)
    if not isinstance(workspace, torch.Tensor) or workspace.device != device or not workspace.is_contiguous():
        raise FAError(1, "workspace must be a contiguous CUDA tensor on %s" % device)
    return workspace


def fa_cache_write(cache, k, v, page_table, seq_lens, cu_seqlens=None, stream=None):
    """Append new rows k, v [T, heads, d] (any strides that keep rows of d contiguous) to the sequences:
    rows cu_seqlens[b] .. cu_seqlens[b+1] - 1 go to sequence b from position seq_lens[b] on; without
    cu_seqlens every sequence gets T / B.  The caller then adds the counts to seq_lens.  A partly filled
    page keeps its scale or takes the larger one of its new tokens; see include/fa.h."""
    desc = _describe(cache)
    device = cache.k.device
    B, stride, P = _check_batch(device, page_table, seq_lens)
    code = _rows(k, "k", 3, device, desc.heads, desc.d)
    if _rows(v, "v", 3, device, desc.heads, desc.d) != code or v.shape != k.shape:
        raise FAError(1, "k and v must share shape and dtype")
    if cu_seqlens is not None and (not isinstance(cu_seqlens, torch.Tensor) or cu_seqlens.device != device
                                   or cu_seqlens.dtype != torch.int32 or cu_seqlens.shape != (B + 1,)
                                   or not cu_seqlens.is_contiguous()):
        raise FAError(1, "cu_seqlens must be a contiguous int32 tensor of B + 1 on %s" % device)
    with _On(device, stream) as on:
        st = fa_cache_write_raw(byref(desc), k.data_ptr(), v.data_ptr(), *_strides(k), *_strides(v),
                                cu_seqlens.data_ptr() if cu_seqlens is not None else None,
                                seq_lens.data_ptr(), page_table.data_ptr(), stride, P, B, k.shape[0],
                                code, on)
    if st != 0:
        raise FAError(st, "fa_cache_write")


def fa_cache_read(cache, page_table, seq_lens, N, dtype=torch.bfloat16, k=None, v=None, stream=None):
    """The first N positions of every sequence as 16-bit k, v [B, heads, N, d], zeros behind seq_lens[b].
    k, v: optional preallocated outputs (their dtype counts then).  Returns (k, v)."""
    desc = _describe(cache)
    device = cache.k.device
    B, stride, P = _check_batch(device, page_table, seq_lens)
    if isinstance(k, torch.Tensor):
        dtype = k.dtype
    elif isinstance(v, torch.Tensor):
        dtype = v.dtype
    if dtype not in _CODES:
        raise FAError(2, "dtype must be float16 or bfloat16, got %s" % dtype)
    if N < 0:
        raise FAError(1, "N must not be negative")
    shape = (B, desc.heads, N, desc.d)
    with _On(device, stream) as on:
        k, v = (torch.empty(shape, dtype=dtype, device=device) if t is None
                else _output(t, name, shape, dtype, device) for t, name in ((k, "k"), (v, "v")))
        st = fa_cache_read_raw(byref(desc), k.data_ptr(), v.data_ptr(), seq_lens.data_ptr(),
                               page_table.data_ptr(), stride, P, B, N, _CODES[dtype], on)
    if st != 0:
        raise FAError(st, "fa_cache_read")
    return k, v


def fa_decode_cache(q, cache, page_table, seq_lens, pages=None, o=None, lse=None, scale=None,
                    causal=False, return_lse=True, workspace=None, stream=None):
    """Decoding attention of q [B, Hq, Nq, d] (1 <= Nq <= 16, Hq a multiple of the cache's heads, any
    strides that keep rows contiguous) to the cache; seq_lens counts the queries' own tokens.  causal
    puts the queries at the end of the sequence.  pages: int32 [B, heads, Nq, slots], the pages that each
    query and KV head reads (``fa_cache_select``), or None for all.  scale defaults to 1/sqrt(d).
    Returns (o, lse); a row without keys has o = 0, lse = -inf."""
    desc = _describe(cache)
    device = cache.k.device
    B, stride, P = _check_batch(device, page_table, seq_lens)
    d = desc.d
    code = _rows(q, "q", 4, device, None, d)
    Hq, Nq = q.shape[1], q.shape[2]
    if q.shape[0] != B or Hq % desc.heads:
        raise FAError(1, "q must be [B, Hq, Nq, d] with Hq a multiple of the cache's heads")
    slots = 0
    if pages is not None:
        slots = pages.shape[-1] if isinstance(pages, torch.Tensor) and pages.dim() else 0
        _output(pages, "pages", (B, desc.heads, Nq, slots), torch.int32, device)
    if scale is None:
        scale = float(d) ** -0.5
    need = fa_decode_cache_workspace_size(B, Hq, desc.heads, Nq, d)
    with _On(device, stream) as on:
        if o is None:
            o = torch.empty((B, Hq, Nq, d), dtype=q.dtype, device=device)
        else:
            _output(o, "o", (B, Hq, Nq, d), q.dtype, device)
        if lse is not None:
            _output(lse, "lse", (B, Hq, Nq), torch.float32, device)
        elif return_lse:
            lse = torch.empty((B, Hq, Nq), dtype=torch.float32, device=device)
        workspace = _workspace(workspace, need, device)
        st = fa_decode_cache_raw(byref(desc), q.data_ptr(), *_strides(q), o.data_ptr(),
                                 lse.data_ptr() if lse is not None else None, seq_lens.data_ptr(),
                                 page_table.data_ptr(), stride, P,
                                 pages.data_ptr() if pages is not None else None, slots,
                                 workspace.data_ptr(), workspace.numel() * workspace.element_size(),
                                 B, Hq, Nq, float(scale), int(bool(causal)), code, on)
    if st != 0:
        raise FAError(st, "fa_decode_cache")
    return o, lse


def fa_cache_select(q, cache, page_table, seq_lens, slots, keep_first=1, keep_last=1, causal=False,
                    pages=None, workspace=None, stream=None):
    """The pages [B, heads, Nq, slots] (int32, ascending, then -1) that q's rows read: the first
    keep_first, the last keep_last and, by the mean keys' scores, the best of the others; all of them
    where there are no more than slots.  Arguments as for fa_decode_cache."""
    desc = _describe(cache)
    device = cache.k.device
    B, stride, P = _check_batch(device, page_table, seq_lens)
    code = _rows(q, "q", 4, device, None, desc.d)
    Hq, Nq = q.shape[1], q.shape[2]
    if q.shape[0] != B or Hq % desc.heads:
        raise FAError(1, "q must be [B, Hq, Nq, d] with Hq a multiple of the cache's heads")
    if slots < 1:
        raise FAError(1, "slots must be at least 1")
    need = fa_cache_select_workspace_size(B, desc.heads, Nq, P)
    shape = (B, desc.heads, Nq, slots)
    with _On(device, stream) as on:
        if pages is None:
            pages = torch.empty(shape, dtype=torch.int32, device=device)
        else:
            _output(pages, "pages", shape, torch.int32, device)
        workspace = _workspace(workspace, need, device)
        st = fa_cache_select_raw(byref(desc), q.data_ptr(), *_strides(q), seq_lens.data_ptr(),
                                 page_table.data_ptr(), stride, P, pages.data_ptr(), slots, keep_first,
                                 keep_last, workspace.data_ptr(),
                                 workspace.numel() * workspace.element_size(), B, Hq, Nq,
                                 int(bool(causal)), code, on)
    if st != 0:
        raise FAError(st, "fa_cache_select")
    return pages
