"""Page tables and slot maps on the GPU (include/fa.h, "Page tables and slot maps from lengths").

    pool = FAPagePool.full(num_pages)
    plan = fa_cache_plan(pool, page_table, seq_lens, new_lens, page, T)
    ...                                                       # write by plan.slots, attend up to plan.ends
    fa_cache_trim(pool, page_table, plan.ends, keep_lens, page)

serve an ``FACache4`` (by slots) and an ``FACache`` (by page table, seq_lens and cu_seqlens) alike.
Lengths, tables and the pool are CUDA tensors that the calls read and write on the device, so that a captured
step follows them.  ``fa_last_device_status`` reports lengths and numbers that are none; a pool that is too
small is no error, and shows in ``plan.ends``.
"""
from typing import NamedTuple

import torch

from ._lib import FAError, fa_cache_plan_raw, fa_cache_trim_raw
from .cache import _check_batch, _elsewhere, _int, _output, _quick, _stream, _there


class FAPagePool(NamedTuple):
    """Free pages: ring int32 [num_pages], and counts int64 [2], the pages taken and given back so far; the free
    ones are ring[x % num_pages] for counts[0] <= x < counts[1]."""
    ring: torch.Tensor
    counts: torch.Tensor

    @classmethod
    def full(cls, num_pages, device="cuda"):
        """All pages free, the lowest first."""
        return cls(torch.arange(num_pages, dtype=torch.int32, device=device),
                   torch.tensor([0, num_pages], dtype=torch.int64, device=device))


class FAPlan(NamedTuple):
    """Of a step's packed rows: where each sequence's begin (cu_seqlens [B + 1]), the sequences' lengths with them
    (ends [B]; the old ones where no room was found), and of each row its position and slot ([T], -1 for none)."""
    cu_seqlens: torch.Tensor
    ends: torch.Tensor
    positions: torch.Tensor
    slots: torch.Tensor


def _check(pool, page_table, seq_lens, other, name, counts):
    if type(pool) is not FAPagePool:
        raise FAError(1, "pool must be an FAPagePool")
    ring, own = pool
    try:
        index = ring.get_device()
        good = (index >= 0 and ring.dtype is torch.int32 and ring.dim() == 1 and ring.is_contiguous()
                and own.get_device() == index and own.dtype is torch.int64 and own.shape == (2,)
                and own.is_contiguous())
    except (AttributeError, TypeError):
        good = False
    if not good:
        raise FAError(1, "an FAPagePool holds contiguous CUDA tensors of one device: ring [num_pages] of int32 and "
                      "counts [2] of int64")
    if counts is not None:
        _output(counts, "counts", (2,), torch.int64, index)
    B, stride, P = _check_batch(index, page_table, seq_lens)
    _output(other, name, (B,), torch.int32, index)
    return index, B, stride, P


def _keep(own, counts):
    """The pool's counts after an empty batch."""
    if counts is not None:
        counts.copy_(own)


def fa_cache_plan(pool, page_table, seq_lens, new_lens, page, T, counts=None, plan=None, stream=None):
    """Find room for new_lens[b] more tokens of each sequence of seq_lens[b]: pages from the pool, in the sequences'
    order, into page_table [B, max_pages], and the ``FAPlan`` of T rows.  A sequence that the free pages do not
    reach for is refused, with all behind it that need any.
    counts: where the pool's counts afterwards go (default: the pool's own; with another tensor the pool stays as it
    was, and another plan may take this one's place).  plan: preallocated outputs.  A batch without sequences takes
    nothing: no row has a slot, and the counts are the pool's.  Returns the plan."""
    if stream is None and plan is None and type(pool) is FAPagePool and (quick := _quick()):
        done = quick.plan(pool, page_table, seq_lens, new_lens, page, T, counts)
        if type(done) is tuple:
            return FAPlan._make(done)
        if done is not None:
            raise FAError(done, "fa_cache_plan")
    index, B, stride, P = _check(pool, page_table, seq_lens, new_lens, "new_lens", counts)
    if _elsewhere(index, stream):
        with _there(index, stream):
            return fa_cache_plan(pool, page_table, seq_lens, new_lens, page, T, counts, plan)
    if _int(T, "T") < 0:
        raise FAError(1, "T must not be negative")
    ring, own = pool
    if plan is None:
        # one allocation, the rows 16-byte aligned in it
        rows, lens = -(-T // 4) * 4, -(-(B + 1) // 4) * 4
        buf = torch.empty(2 * rows + 2 * lens, dtype=torch.int32, device=ring.device)
        plan = FAPlan(buf[2 * rows:2 * rows + B + 1], buf[2 * rows + lens:2 * rows + lens + B], buf[:T], buf[rows:rows + T])
    elif type(plan) is FAPlan:
        for t, name, n in zip(plan, FAPlan._fields, (B + 1, B, T, T)):
            _output(t, "plan." + name, (n,), torch.int32, index)
    else:
        raise FAError(1, "plan must be an FAPlan")
    out = own if counts is None else counts
    st = fa_cache_plan_raw(ring.data_ptr(), _int(ring.shape[0], "num_pages"), own.data_ptr(), page_table.data_ptr(),
                           stride, P, seq_lens.data_ptr(), new_lens.data_ptr(), plan.cu_seqlens.data_ptr(),
                           plan.ends.data_ptr(), plan.positions.data_ptr(), plan.slots.data_ptr(), out.data_ptr(),
                           _int(page, "page"), B, T, _stream(index))
    if st != 0:
        raise FAError(st, "fa_cache_plan")
    if B == 0:  # the library writes nothing
        plan.cu_seqlens.zero_()
        plan.positions.fill_(-1)
        plan.slots.fill_(-1)
        _keep(own, counts)
    return plan


def fa_cache_trim(pool, page_table, seq_lens, keep_lens, page, counts=None, stream=None):
    """Cut sequences of seq_lens[b] tokens to keep_lens[b] (0: done) and give the pages behind back to the pool.
    The caller's lengths become keep_lens afterwards.  counts: as for ``fa_cache_plan``."""
    if stream is None and type(pool) is FAPagePool and (quick := _quick()):
        done = quick.trim(pool, page_table, seq_lens, keep_lens, page, counts)
        if done is not None:
            if done:
                raise FAError(done, "fa_cache_trim")
            return
    index, B, stride, P = _check(pool, page_table, seq_lens, keep_lens, "keep_lens", counts)
    if _elsewhere(index, stream):
        with _there(index, stream):
            return fa_cache_trim(pool, page_table, seq_lens, keep_lens, page, counts)
    ring, own = pool
    out = own if counts is None else counts
    st = fa_cache_trim_raw(ring.data_ptr(), _int(ring.shape[0], "num_pages"), own.data_ptr(), page_table.data_ptr(),
                           stride, P, seq_lens.data_ptr(), keep_lens.data_ptr(), out.data_ptr(), _int(page, "page"), B,
                           _stream(index))
    if st != 0:
        raise FAError(st, "fa_cache_trim")
    if B == 0:  # the library writes nothing
        _keep(own, counts)
