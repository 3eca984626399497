"""The 4-bit paged KV cache on torch tensors (include/fa.h, "The 4-bit paged KV cache").

    cache = FACache4.empty(num_pages, heads, page, d)
    plan = fa_cache_plan(pool, page_table, seq_lens, new_lens, page, T)
    fa_cache4_write(cache, k, v, plan.slots)                   # k, v [T, heads, d]
    o, lse = fa_decode_cache4(q, cache, page_table, plan.ends)  # q [B, Hq, Nq, d]

Page tables and lengths are those of the 8-bit cache, and so is what the calls do with bad
ones.  Every token stands by itself (sixteen of its channels share a scale), so that rows go
to any slots, in any order, and writing changes nothing that was written before.
"""
from struct import Struct
from typing import NamedTuple

import torch

from ._lib import (FAError, fa_cache4_read_raw, fa_cache4_write_raw, fa_decode_cache4_raw,
                   fa_decode_cache4_workspace_size)
from .cache import _CODES, _check_batch, _code, _elsewhere, _int, _output, _quick, _stream, _there, _workspace


class FACache4(NamedTuple):
    """The buffer of a cache, uint8 [num_pages, heads, page, 9 d / 8].  The last two dimensions are one
    block of bytes: ``parts`` shows what lies where.  Nothing is kept beside it."""
    data: torch.Tensor

    @classmethod
    def empty(cls, num_pages, heads, page, d, device="cuda"):
        """A cache with nothing in it (its memory is not initialised)."""
        if d % 32 or d < 32:
            raise FAError(2, "d must be 32, 64, 96 or 128, got %s" % d)
        return cls(torch.empty((num_pages, heads, page, d // 8 * 9), dtype=torch.uint8, device=device))

    def parts(self):
        """Views of the codes of K [num_pages, heads, page, d / 2] (channel 2 c in the low half of byte c), its
        scales [.., page, d / 16] (a byte is an fp16's bits 14 .. 7), and the same of V."""
        page, d = self.data.shape[2], self.data.shape[3] // 9 * 8
        flat, sizes = self.data.flatten(2), [page * d // 2, page * d // 16] * 2
        return tuple(x.unflatten(-1, (page, -1)) for x in flat.split(sizes, -1))


# fa_cache4_t of include/fa.h: a pointer, four ints
_DESC = Struct("Q4i").pack


def _describe(cache):
    """The checked fa_cache4_t of a cache (as bytes, for ctypes), its heads, head dimension and device number."""
    if type(cache) is not FACache4:
        raise FAError(1, "cache must be an FACache4")
    data = cache.data
    try:
        index = data.get_device()
        num_pages, heads, page, wide = data.shape
        good = index >= 0 and data.dtype is torch.uint8 and data.is_contiguous() and wide % 36 == 0
    except (AttributeError, TypeError, ValueError):
        good = False
    if not good:
        raise FAError(1, "an FACache4 holds one contiguous CUDA tensor of uint8, [num_pages, heads, page, 9 d / 8]")
    d = wide // 9 * 8
    return _DESC(data.data_ptr(), _int(num_pages, "num_pages"), heads, page, d), heads, d, index


def fa_cache4_write(cache, k, v, slots, stream=None):
    """Write rows k, v [T, heads, d] (any strides that keep rows of d contiguous) to slots [T] (int32: page
    number * page + place in the page, as ``fa_cache_plan`` gives them; rows with a negative one are left out)."""
    if stream is None and type(cache) is FACache4 and (quick := _quick()):
        done = quick.write4(cache, k, v, slots)
        if done is not None:
            if done:
                raise FAError(done, "fa_cache4_write")
            return
    desc, heads, d, index = _describe(cache)
    if _elsewhere(index, stream):
        with _there(index, stream):
            return fa_cache4_write(cache, k, v, slots)
    code = _code(k, "k", 3, index, d)
    shape = k.shape
    if _code(v, "v", 3, index, d) != code or v.shape != shape or shape[1] != heads:
        raise FAError(1, "k and v must be [T, heads, d] of one dtype")
    _output(slots, "slots", (shape[0],), torch.int32, index)
    kt, kh, _ = k.stride()
    vt, vh, _ = v.stride()
    st = fa_cache4_write_raw(desc, k.data_ptr(), v.data_ptr(), kt, kh, vt, vh, slots.data_ptr(), _int(shape[0], "T"),
                             code, _stream(index))
    if st != 0:
        raise FAError(st, "fa_cache4_write")


def fa_cache4_read(cache, page_table, seq_lens, N, dtype=torch.bfloat16, k=None, v=None, stream=None):
    """The first N positions of every sequence as 16-bit k, v [B, heads, N, d], exact in either type, zeros behind
    seq_lens[b] (which are no mask: attention that sees them counts them as keys of score 0).
    k, v: optional preallocated outputs (their dtype counts then).  Returns (k, v)."""
    if stream is None and type(cache) is FACache4 and dtype in _CODES and (quick := _quick()):
        given = k if k is not None else v
        done = quick.read4(cache, page_table, seq_lens, N,
                           (dtype if given is None else getattr(given, "dtype", None)) is torch.float16, k, v)
        if type(done) is tuple:
            return done
        if done is not None:
            raise FAError(done, "fa_cache4_read")
    desc, heads, d, index = _describe(cache)
    if _elsewhere(index, stream):
        with _there(index, stream):
            return fa_cache4_read(cache, page_table, seq_lens, N, dtype, k, v)
    B, stride, P = _check_batch(index, page_table, seq_lens)
    given = k if k is not None else v
    if isinstance(given, torch.Tensor):
        dtype = given.dtype
    code = _CODES.get(dtype)
    if code is None:
        raise FAError(2, "dtype must be float16 or bfloat16, got %s" % dtype)
    if _int(N, "N") < 0:
        raise FAError(1, "N must not be negative")
    shape, device = (B, heads, N, d), cache.data.device
    k = torch.empty(shape, dtype=dtype, device=device) if k is None else _output(k, "k", shape, dtype, index)
    v = torch.empty(shape, dtype=dtype, device=device) if v is None else _output(v, "v", shape, dtype, index)
    st = fa_cache4_read_raw(desc, k.data_ptr(), v.data_ptr(), seq_lens.data_ptr(), page_table.data_ptr(), stride, P, B,
                            N, code, _stream(index))
    if st != 0:
        raise FAError(st, "fa_cache4_read")
    return k, v


def fa_decode_cache4(q, cache, page_table, seq_lens, o=None, lse=None, scale=None, causal=False, return_lse=True,
                     workspace=None, stream=None):
    """Decoding attention of q [B, Hq, Nq, d] (1 <= Nq <= 16, Hq a multiple of the cache's heads, any strides that
    keep rows contiguous) to the cache; seq_lens counts the queries' own tokens.  causal puts the queries at the
    end of the sequence.  scale defaults to 1/sqrt(d).  Returns (o, lse); a row without keys has o = 0,
    lse = -inf.
    The lengths are on the device: how the work is shared out follows the page table's width.  Where the longest
    sequence is known to be short, its first columns are faster: page_table[:, :pages of the longest]."""
    if stream is None and type(cache) is FACache4 and (quick := _quick()):
        done = quick.decode4(q, cache, page_table, seq_lens, o, lse, scale if scale is None else float(scale),
                             True if causal else False, True if return_lse else False, workspace)
        if type(done) is tuple:
            return done
        if done is not None:
            raise FAError(done, "fa_decode_cache4")
    desc, heads, d, index = _describe(cache)
    if _elsewhere(index, stream):
        with _there(index, stream):
            return fa_decode_cache4(q, cache, page_table, seq_lens, o, lse, scale, causal, return_lse, workspace)
    B, stride, P = _check_batch(index, page_table, seq_lens)
    code = _code(q, "q", 4, index, d)
    shape = q.shape
    Bq, Hq, Nq, _ = shape
    if Bq != B or _int(Hq, "Hq") % heads:
        raise FAError(1, "q must be [B, Hq, Nq, d] with Hq a multiple of the cache's heads")
    _int(Nq, "Nq")
    if scale is None:
        scale = float(d) ** -0.5
    device = cache.data.device
    if o is None:
        o = torch.empty(shape, dtype=q.dtype, device=device)
    else:
        _output(o, "o", shape, q.dtype, index)
    if lse is not None:
        _output(lse, "lse", (B, Hq, Nq), torch.float32, index)
    elif return_lse:
        lse = torch.empty((B, Hq, Nq), dtype=torch.float32, device=device)
    if workspace is None:
        need = fa_decode_cache4_workspace_size(B, Hq, heads, Nq, d)
        workspace = torch.empty(max(need, 16), dtype=torch.uint8, device=device)
    else:
        _workspace(workspace, index)
    sb, sh, sn, _ = q.stride()
    st = fa_decode_cache4_raw(desc, q.data_ptr(), sb, sh, sn, o.data_ptr(), lse.data_ptr() if lse is not None else None,
                              seq_lens.data_ptr(), page_table.data_ptr(), stride, P, workspace.data_ptr(),
                              workspace.nbytes, B, Hq, Nq, scale, 1 if causal else 0, code, _stream(index))
    if st != 0:
        raise FAError(st, "fa_decode_cache4")
    return o, lse
