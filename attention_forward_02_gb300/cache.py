"""The 8-bit paged KV cache on torch tensors (include/fa.h, "The 8-bit paged KV cache").

    cache = FACache.empty(num_pages, heads, page, d)          # e4m3, or dtype=torch.int8
    fa_cache_write(cache, k, v, page_table, seq_lens)         # k, v [T, heads, d]
    seq_lens += T // B
    o, lse = fa_decode_cache(q, cache, page_table, seq_lens)  # q [B, Hq, Nq, d]

or, over the best pages of a long cache,

    pages = fa_cache_select(q, cache, page_table, seq_lens, slots)
    o, lse = fa_decode_cache(q, cache, page_table, seq_lens, pages=pages)

and ``k, v = fa_cache_read(cache, page_table, seq_lens, N)`` in 16 bits, for
``fa_fwd`` with ``causal`` or, each sequence cut to its length, ``fa_decode``.
``page_table`` [B, max_pages] and ``seq_lens`` [B] are int32 CUDA tensors; the calls
read them on the device, so a captured graph replays with whatever they hold then.
What they hold cannot be checked by the call: a page number outside the cache is
left out, a length outside the page table is cut to it (and nothing is written for a
negative one), and ``fa_last_device_status`` reports either.
"""
import importlib.machinery
import importlib.util
import os
from ctypes import c_void_p, cast
from struct import Struct
from typing import NamedTuple, Optional

import torch

from ._lib import (FA_BF16, FA_E4M3, FA_FP16, FA_INT8, FAError, fa_cache_read_raw,
                   fa_cache_select_raw, fa_cache_select_workspace_size, fa_cache_write_raw,
                   fa_decode_cache_raw, fa_decode_cache_workspace_size, load)
from .build import BINDING, BINDING_NAME

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


# The CPython module of csrc/fa_cache_py.cpp goes through a usual call's checks and allocations in less
# time than Python does; it hands back (None) what is not usual, and the functions below see to that.
_module = None   # the module; False where there is none that can be used
_bound = None    # the library whose addresses it holds


def _load_module():
    """The module, if it was built, loads, and was built for this torch; else False."""
    if not os.path.exists(BINDING):
        return False
    try:
        loader = importlib.machinery.ExtensionFileLoader(BINDING_NAME, BINDING)
        module = importlib.util.module_from_spec(importlib.util.spec_from_loader(BINDING_NAME, loader))
        loader.exec_module(module)
    except (ImportError, OSError):
        return False
    return module if getattr(module, "torch", None) == str(torch.__version__) else False


def _quick():
    global _module, _bound
    lib = load()
    if lib is not _bound:
        if _module is None:
            _module = _load_module()
        if _module and _module.abi != lib.fa_abi_version():
            _module = False
        if _module:
            _module.bind(*(cast(f, c_void_p).value for f in (
                lib.fa_cache_write, lib.fa_cache_read, lib.fa_decode_cache, lib.fa_decode_cache_workspace_size,
                lib.fa_cache_select, lib.fa_cache_select_workspace_size)))
        _bound = lib
    return _module


# fa_cache_t of include/fa.h: six pointers, five ints
_DESC = Struct("6Q5i4x").pack


def _describe(cache):
    """The checked fa_cache_t of a cache (as bytes, for ctypes), its KV heads, head dimension and device number."""
    if type(cache) is not FACache:
        raise FAError(1, "cache must be an FACache")
    try:
        k, v, ks, vs, mean, ms = cache
        shape, dtype, index = k.shape, k.dtype, k.get_device()
        num_pages, heads, page, d = shape
        pair = (num_pages, heads)
        fmt = _FORMATS[dtype]
        good = (index >= 0 and k.is_contiguous()
                and v.get_device() == index and v.shape == shape and v.dtype is dtype and v.is_contiguous()
                and ks.get_device() == index and ks.shape == pair and ks.dtype is torch.float32
                and ks.is_contiguous()
                and vs.get_device() == index and vs.shape == pair and vs.dtype is torch.float32
                and vs.is_contiguous())
        mp = sp = 0
        if good and (mean is not None or ms is not None):
            good = (mean.get_device() == index and mean.shape == (num_pages, heads, d)
                    and mean.dtype is torch.int8 and mean.is_contiguous()
                    and ms.get_device() == index and ms.shape == pair and ms.dtype is torch.float32
                    and ms.is_contiguous())
            mp, sp = mean.data_ptr(), ms.data_ptr()
    except (AttributeError, KeyError, TypeError, ValueError):
        good = False
    if not good:
        raise FAError(1, "an FACache holds contiguous CUDA tensors of one device: k, v [num_pages, heads, page, d] "
                      "of float8_e4m3fn or int8, k_scale, v_scale [num_pages, heads] of float32 and, both or "
                      "neither, k_mean [num_pages, heads, d] of int8, k_mean_scale like k_scale")
    return (_DESC(k.data_ptr(), v.data_ptr(), ks.data_ptr(), vs.data_ptr(), mp, sp, num_pages, heads, page, d, fmt),
            heads, d, index)


def _int(x, name):
    """A whole number as the C ABI takes it: ctypes would cut it to its low 32 bits."""
    if not -2 ** 31 <= x < 2 ** 31:
        raise FAError(1, "%s must fit 32 bits, got %s" % (name, x))
    return x


def _check_batch(index, page_table, seq_lens):
    """Sequences, distance of the page table's rows, its columns."""
    try:
        B, P = page_table.shape
        good = (seq_lens.shape == (B,) and page_table.get_device() == index and seq_lens.get_device() == index
                and page_table.dtype is torch.int32 and seq_lens.dtype is torch.int32
                and (P <= 1 or page_table.stride(1) == 1) and seq_lens.is_contiguous())
    except (AttributeError, TypeError, ValueError):
        good = False
    if not good:
        raise FAError(1, "page_table [B, max_pages] and seq_lens [B] must be int32 tensors on the cache's device, "
                      "their last dimension contiguous")
    return _int(B, "B"), page_table.stride(0) if B > 1 else P, _int(P, "max_pages")


def _code(t, name, dim, index, d):
    """Checks an input whose rows of d values are contiguous; returns its type's code."""
    try:
        shape = t.shape
        good = (len(shape) == dim and shape[-1] == d and t.get_device() == index
                and (t.stride(-1) == 1 or t.numel() == 0))
    except (AttributeError, TypeError, IndexError):
        good = False
    if not good:
        raise FAError(1, "%s must be a %d-dimensional tensor of rows of %d contiguous values on the cache's device"
                      % (name, dim, d))
    code = _CODES.get(t.dtype)
    if code is None:
        raise FAError(2, "%s must be float16 or bfloat16, got %s" % (name, t.dtype))
    return code


def _output(t, name, shape, dtype, index):
    if (not isinstance(t, torch.Tensor) or t.get_device() != index or t.shape != shape or t.dtype != dtype
            or not t.is_contiguous()):
        raise FAError(1, "%s must be a contiguous tensor %s of %s on the cache's device" % (name, shape, dtype))
    return t


def _elsewhere(index, stream):
    """Whether a call has to go to a device or stream that is not the current one."""
    return stream is not None or torch.cuda.current_device() != index


def _there(index, stream):
    """The context for it.  What a call allocates inside belongs to that stream."""
    if stream is None:
        return torch.cuda.device(index)
    if stream.device.index != index:
        raise FAError(1, "the stream must be one of the cache's device")
    return torch.cuda.stream(stream)


def _stream(index):
    """The current stream's handle."""
    return torch.cuda.current_stream(index).cuda_stream


# the same without a Stream object, where this torch has it: 0.1 us instead of 2
_stream = getattr(torch._C, "_cuda_getCurrentRawStream", _stream)


def _workspace(workspace, index):
    if (not isinstance(workspace, torch.Tensor) or workspace.get_device() != index
            or not workspace.is_contiguous()):
        raise FAError(1, "workspace must be a contiguous tensor on the cache's device")
    return workspace


def fa_cache_write(cache, k, v, page_table, seq_lens, cu_seqlens=None, stream=None):
    """Append new rows k, v [T, heads, d] (any strides that keep rows of d contiguous) to the sequences:
    rows cu_seqlens[b] .. cu_seqlens[b+1] - 1 go to sequence b from position seq_lens[b] on; without
    cu_seqlens every sequence gets T / B.  The caller then adds the counts to seq_lens.  A partly filled
    page keeps its scale or takes the larger one of its new tokens; see include/fa.h."""
    if stream is None and type(cache) is FACache and (quick := _quick()):
        done = quick.write(cache, k, v, page_table, seq_lens, cu_seqlens)
        if done is not None:
            if done:
                raise FAError(done, "fa_cache_write")
            return
    desc, heads, d, index = _describe(cache)
    if _elsewhere(index, stream):
        with _there(index, stream):
            return fa_cache_write(cache, k, v, page_table, seq_lens, cu_seqlens)
    B, stride, P = _check_batch(index, page_table, seq_lens)
    code = _code(k, "k", 3, index, d)
    shape = k.shape
    if _code(v, "v", 3, index, d) != code or v.shape != shape or shape[1] != heads:
        raise FAError(1, "k and v must be [T, heads, d] of one dtype")
    cu = None
    if cu_seqlens is not None:
        _output(cu_seqlens, "cu_seqlens", (B + 1,), torch.int32, index)
        cu = cu_seqlens.data_ptr()
    kt, kh, _ = k.stride()
    vt, vh, _ = v.stride()
    st = fa_cache_write_raw(desc, k.data_ptr(), v.data_ptr(), kt, kh, vt, vh, cu, seq_lens.data_ptr(),
                            page_table.data_ptr(), stride, P, B, _int(shape[0], "T"), code, _stream(index))
    if st != 0:
        raise FAError(st, "fa_cache_write")


def fa_cache_read(cache, page_table, seq_lens, N, dtype=torch.bfloat16, k=None, v=None, stream=None):
    """The first N positions of every sequence as 16-bit k, v [B, heads, N, d], zeros behind seq_lens[b]
    (which are no mask: attention that sees them counts them as keys of score 0).
    k, v: optional preallocated outputs (their dtype counts then).  Returns (k, v)."""
    if stream is None and type(cache) is FACache and dtype in _CODES and (quick := _quick()):
        given = k if k is not None else v
        done = quick.read(cache, page_table, seq_lens, N,
                          (dtype if given is None else getattr(given, "dtype", None)) is torch.float16, k, v)
        if type(done) is tuple:
            return done
        if done is not None:
            raise FAError(done, "fa_cache_read")
    desc, heads, d, index = _describe(cache)
    if _elsewhere(index, stream):
        with _there(index, stream):
            return fa_cache_read(cache, page_table, seq_lens, N, dtype, k, v)
    B, stride, P = _check_batch(index, page_table, seq_lens)
    given = k if k is not None else v
    if isinstance(given, torch.Tensor):
        dtype = given.dtype
    code = _CODES.get(dtype)
    if code is None:
        raise FAError(2, "dtype must be float16 or bfloat16, got %s" % dtype)
    if _int(N, "N") < 0:
        raise FAError(1, "N must not be negative")
    shape = (B, heads, N, d)
    device = cache.k.device
    k = torch.empty(shape, dtype=dtype, device=device) if k is None else _output(k, "k", shape, dtype, index)
    v = torch.empty(shape, dtype=dtype, device=device) if v is None else _output(v, "v", shape, dtype, index)
    st = fa_cache_read_raw(desc, k.data_ptr(), v.data_ptr(), seq_lens.data_ptr(), page_table.data_ptr(), stride, P, B,
                           N, code, _stream(index))
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
    if stream is None and type(cache) is FACache and (quick := _quick()):
        done = quick.decode(q, cache, page_table, seq_lens, pages, o, lse, scale if scale is None else float(scale),
                            True if causal else False, True if return_lse else False, workspace)
        if type(done) is tuple:
            return done
        if done is not None:
            raise FAError(done, "fa_decode_cache")
    desc, heads, d, index = _describe(cache)
    if _elsewhere(index, stream):
        with _there(index, stream):
            return fa_decode_cache(q, cache, page_table, seq_lens, pages, o, lse, scale, causal, return_lse, workspace)
    B, stride, P = _check_batch(index, page_table, seq_lens)
    code = _code(q, "q", 4, index, d)
    shape = q.shape
    Bq, Hq, Nq, _ = shape
    if Bq != B or _int(Hq, "Hq") % heads:
        raise FAError(1, "q must be [B, Hq, Nq, d] with Hq a multiple of the cache's heads")
    _int(Nq, "Nq")
    slots, listed = 0, None
    if pages is not None:
        slots = _int(pages.shape[-1], "slots") if isinstance(pages, torch.Tensor) and pages.dim() else 0
        listed = _output(pages, "pages", (B, heads, Nq, slots), torch.int32, index).data_ptr()
    if scale is None:
        scale = float(d) ** -0.5
    device = cache.k.device
    if o is None:
        o = torch.empty(shape, dtype=q.dtype, device=device)
    else:
        _output(o, "o", shape, q.dtype, index)
    if lse is not None:
        _output(lse, "lse", (B, Hq, Nq), torch.float32, index)
    elif return_lse:
        lse = torch.empty((B, Hq, Nq), dtype=torch.float32, device=device)
    if workspace is None:
        need = fa_decode_cache_workspace_size(B, Hq, heads, Nq, d)
        workspace = torch.empty(max(need, 16), dtype=torch.uint8, device=device)
    else:
        _workspace(workspace, index)
    sb, sh, sn, _ = q.stride()
    st = fa_decode_cache_raw(desc, q.data_ptr(), sb, sh, sn, o.data_ptr(), lse.data_ptr() if lse is not None else None,
                             seq_lens.data_ptr(), page_table.data_ptr(), stride, P, listed, slots,
                             workspace.data_ptr(), workspace.nbytes, B, Hq, Nq, scale, 1 if causal else 0, code,
                             _stream(index))
    if st != 0:
        raise FAError(st, "fa_decode_cache")
    return o, lse


def fa_cache_select(q, cache, page_table, seq_lens, slots, keep_first=1, keep_last=1, causal=False,
                    pages=None, workspace=None, stream=None):
    """The pages [B, heads, Nq, slots] (int32, ascending, then -1) that q's rows read: the first
    keep_first, the last keep_last and, by the mean keys' scores, the best of the others; all of them
    where there are no more than slots.  Arguments as for fa_decode_cache."""
    if stream is None and type(cache) is FACache and (quick := _quick()):
        done = quick.select(q, cache, page_table, seq_lens, slots, keep_first, keep_last,
                            True if causal else False, pages, workspace)
        if type(done) is int:
            raise FAError(done, "fa_cache_select")
        if done is not None:
            return done
    desc, heads, d, index = _describe(cache)
    if _elsewhere(index, stream):
        with _there(index, stream):
            return fa_cache_select(q, cache, page_table, seq_lens, slots, keep_first, keep_last, causal, pages, workspace)
    B, stride, P = _check_batch(index, page_table, seq_lens)
    code = _code(q, "q", 4, index, d)
    Bq, Hq, Nq, _ = q.shape
    if Bq != B or _int(Hq, "Hq") % heads:
        raise FAError(1, "q must be [B, Hq, Nq, d] with Hq a multiple of the cache's heads")
    _int(Nq, "Nq")
    if Hq == 0 and B > 0:
        raise FAError(1, "pages are chosen by their scores with query heads, and q has none")
    if _int(slots, "slots") < 1:
        raise FAError(1, "slots must be at least 1")
    _int(keep_first, "keep_first"), _int(keep_last, "keep_last")
    shape = (B, heads, Nq, slots)
    device = cache.k.device
    if pages is None:
        pages = torch.empty(shape, dtype=torch.int32, device=device)
    else:
        _output(pages, "pages", shape, torch.int32, index)
    if workspace is None:
        need = fa_cache_select_workspace_size(B, heads, Nq, P)
        workspace = torch.empty(max(need, 16), dtype=torch.uint8, device=device)
    else:
        _workspace(workspace, index)
    sb, sh, sn, _ = q.stride()
    st = fa_cache_select_raw(desc, q.data_ptr(), sb, sh, sn, seq_lens.data_ptr(), page_table.data_ptr(), stride, P,
                             pages.data_ptr(), slots, keep_first, keep_last, workspace.data_ptr(), workspace.nbytes, B,
                             Hq, Nq, 1 if causal else 0, code, _stream(index))
    if st != 0:
        raise FAError(st, "fa_cache_select")
    return pages
