"""Rotary positions of query and key rows on torch tensors (include/fa.h, "Rotary positions").

    rope = FARope.new(128)                                    # or part of the head, interleaved, scaled
    q, k = fa_rope(q, k, rope, positions)                     # [T, heads, d] or [B, heads, N, d]
    dq, dk = fa_rope(dq, dk, rope, positions, backward=True)  # gradients of turned rows to those before
"""
import math
from ctypes import byref
from functools import lru_cache
from typing import NamedTuple

import torch

from ._lib import FAError, RopeDesc, RopeRows, fa_rope_raw
from .cache import _CODES, _elsewhere, _int, _quick, _stream, _there


@lru_cache(maxsize=8)
def _per_turn(bits):
    """2^bits / (2 pi), cut to a whole number."""
    one = 1 << (bits + 64)

    def arctan(n):  # of 1 / n
        total, term, k = 0, one // n, 1
        while term:
            total += term // k if k % 4 == 1 else -(term // k)
            term //= n * n
            k += 2
        return total

    pi = 4 * (4 * arctan(5) - arctan(239))  # Machin's formula, 64 bits to spare
    return one * (1 << bits) // (2 * pi)


def _turns(x):
    """x radians as turns times 2^64, rounded to a whole number, modulo 2^64 in two's complement."""
    mantissa, exponent = math.frexp(x)  # x = whole * 2^down, whole of 53 bits
    whole, down = int(math.ldexp(mantissa, 53)), exponent - 53
    bits = 256 + max(0, exponent + 255) // 256 * 256  # 128 and more behind the last one that counts
    shift = bits - 64 - down
    turns = (whole * _per_turn(bits) + (1 << (shift - 1))) >> shift
    return (turns + 2 ** 63) % 2 ** 64 - 2 ** 63


def _scaled(rot, base, scaling, factor, trained, fast, slow):
    """Radians a position of each pair, and the factor on the turned channels."""
    if not (math.isfinite(base) and base > 0 and math.isfinite(factor) and factor > 0):
        raise FAError(1, "base and factor must be positive")
    if scaling == "base":
        base *= factor ** (rot / max(2, rot - 2))
    w = [base ** (-2.0 * i / rot) for i in range(rot // 2)]
    if scaling is None or scaling == "base":
        return w, 1.0
    if scaling == "linear":
        return [x / factor for x in w], 1.0
    if scaling not in ("yarn", "bands"):
        raise FAError(1, "scaling must be None, 'linear', 'base', 'yarn' or 'bands', got %r" % (scaling,))
    if not (trained and trained > 0 and fast > slow > 0):
        raise FAError(1, "scaling %r needs trained > 0 and fast > slow > 0" % scaling)
    if scaling == "bands":
        # by the turns of a pair over the trained positions: `slow` and fewer are stretched, `fast` and more not
        turns = [trained * x / (2 * math.pi) for x in w]
        keep = [min(1.0, max(0.0, (t - slow) / (fast - slow))) for t in turns]
        return [x * y + x / factor * (1 - y) for x, y in zip(w, keep)], 1.0
    # by the pair's number, between those that turn `fast` and `slow` times over the trained positions
    at = [rot * math.log(trained / (t * 2 * math.pi)) / (2 * math.log(base)) for t in (fast, slow)]
    lo, hi = max(0, math.floor(at[0])), min(rot - 1, math.ceil(at[1]))
    part = [min(1.0, max(0.0, (i - lo) / max(hi - lo, 0.001))) for i in range(rot // 2)]
    return ([x * (1 - y) + x / factor * y for x, y in zip(w, part)],
            0.1 * math.log(factor) + 1.0 if factor > 1 else 1.0)


class FARope(NamedTuple):
    """How positions turn heads: turns int64 [pairs], the fraction of a turn that a position turns each pair by,
    times 2^64 and rounded (two's complement); whether neighbouring channels pair, or those half the turned part apart; and
    a factor on the turned channels.  Nothing is kept beside them."""
    turns: torch.Tensor
    interleaved: bool = False
    factor: float = 1.0

    @classmethod
    def new(cls, rot, base=10000.0, interleaved=False, scaling=None, factor=8.0, trained=None, fast=32.0, slow=1.0,
            radians=None, device="cuda"):
        """Turning the first rot channels (a multiple of 8), pair i by base^(-2 i / rot) a position.  scaling, for
        contexts `factor` times the trained ones: "linear" (every pair slower by it), "base" (the base grows, so that
        the slowest pair is slower by it and the fastest stays), "bands" or "yarn" (pairs that turn `slow` times and
        fewer over `trained` positions slower by it, those that turn `fast` times and more as they were, the others in
        between, by their turns or by their number; "yarn" scales the turned channels too).  radians: the rot / 2
        angles a position themselves."""
        if not isinstance(rot, int) or rot < 8 or rot % 8:
            raise FAError(2, "rot must be a multiple of 8, got %s" % (rot,))
        on_channels = 1.0
        if radians is None:
            try:
                radians, on_channels = _scaled(rot, float(base), scaling, float(factor), trained, float(fast), float(slow))
            except (OverflowError, ValueError, ZeroDivisionError):
                raise FAError(1, "these numbers give no frequencies") from None
            if not all(math.isfinite(x) for x in (*radians, on_channels)):
                raise FAError(1, "these numbers give no finite frequencies")
        else:
            radians = [float(x) for x in radians]
            if len(radians) != rot // 2 or not all(math.isfinite(x) for x in radians):
                raise FAError(1, "radians must be rot / 2 finite numbers")
        return cls(torch.tensor([_turns(x) for x in radians], dtype=torch.int64, device=device), bool(interleaved), on_channels)


def _rows(x, name, index, out, like):
    """The checked RopeRows of x and its output, the output, and the type's code."""
    try:
        dim, shape = x.dim(), x.shape
        good = dim in (3, 4) and x.get_device() == index and (x.stride(-1) == 1 or x.numel() == 0)
    except (AttributeError, TypeError, IndexError):
        good = False
    if not good:
        raise FAError(1, "%s must be [T, heads, d] or [B, heads, N, d], rows of contiguous values, on one CUDA device"
                      % name)
    code = _CODES.get(x.dtype)
    if code is None:
        raise FAError(2, "%s must be float16 or bfloat16, got %s" % (name, x.dtype))
    if like is not None and (dim != like.dim() or x.dtype != like.dtype or shape[-1] != like.shape[-1]
                             or shape[0] != like.shape[0] or (dim == 4 and shape[2] != like.shape[2])):
        raise FAError(1, "q and k must be of one dtype, and differ in their heads only")
    if out is None:
        out = torch.empty(shape, dtype=x.dtype, device=x.device)
    elif (not isinstance(out, torch.Tensor) or out.shape != shape or out.dtype != x.dtype
          or out.get_device() != index or (out.stride(-1) != 1 and out.numel() != 0)):
        raise FAError(1, "%s_out must be shaped and typed like %s, rows of contiguous values" % (name, name))
    if dim == 3:
        (xn, xh, _), (yn, yh, _) = x.stride(), out.stride()
        xb = yb = 0
        heads = shape[1]
    else:
        (xb, xh, xn, _), (yb, yh, yn, _) = x.stride(), out.stride()
        heads = shape[1]
    return RopeRows(x.data_ptr(), out.data_ptr(), xb, xh, xn, yb, yh, yn, _int(heads, "heads")), out, code


def fa_rope(q, k, rope, positions=None, backward=False, q_out=None, k_out=None, stream=None):
    """q and k (k may be None) turned to their positions: packed tokens [T, heads, d], or [B, heads, N, d] as
    ``fa_fwd`` takes them, any strides that keep rows of d contiguous.  positions: int32 [T], or [N] or [B, N];
    None counts rows from 0; a row at a negative one stays as it is.  backward: gradients with respect to turned
    rows in, those with respect to the rows before out.  q_out, k_out: optional outputs, q and k themselves among
    them.  Returns (q, k) turned; computed in fp32 and rounded once."""
    if stream is None and type(rope) is FARope and (quick := _quick()):
        done = quick.rope(q, k, rope, positions, True if backward else False, q_out, k_out)
        if type(done) is tuple:
            return done
        if done is not None:
            raise FAError(done, "fa_rope")
    index = q.get_device() if isinstance(q, torch.Tensor) else -1
    if index < 0:
        raise FAError(1, "q must be a CUDA tensor")
    if _elsewhere(index, stream):
        with _there(index, stream):
            return fa_rope(q, k, rope, positions, backward, q_out, k_out)
    if type(rope) is not FARope:
        raise FAError(1, "rope must be an FARope")
    turns = rope.turns
    if (not isinstance(turns, torch.Tensor) or turns.get_device() != index or turns.dtype is not torch.int64
            or turns.dim() != 1 or not turns.is_contiguous()):
        raise FAError(1, "rope.turns must be a contiguous tensor [pairs] of int64 on q's device")
    rows_q, q_out, code = _rows(q, "q", index, q_out, None)
    rows_k = None
    if k is not None:
        rows_k, k_out, _ = _rows(k, "k", index, k_out, q)
    elif k_out is not None:
        raise FAError(1, "k_out without k")
    if q.dim() == 3:
        B, N = 1, q.shape[0]
        shapes = ((N,),)
    else:
        B, N = q.shape[0], q.shape[2]
        shapes = ((N,), (B, N))
    at, stride = None, 0
    if positions is not None:
        if (not isinstance(positions, torch.Tensor) or positions.get_device() != index
                or positions.dtype is not torch.int32 or positions.shape not in shapes
                or (positions.stride(-1) != 1 and N > 1)):
            raise FAError(1, "positions must be int32 on q's device, %s, the last dimension contiguous"
                          % " or ".join(str(list(s)) for s in shapes))
        at = positions.data_ptr()
        if positions.dim() == 2:
            stride = positions.stride(0)
    desc = RopeDesc(turns.data_ptr(), turns.shape[0], 1 if rope.interleaved else 0, rope.factor)
    st = fa_rope_raw(byref(desc), byref(rows_q), byref(rows_k) if rows_k is not None else None, at, stride,
                     _int(B, "B"), _int(N, "N"), q.shape[-1], 1 if backward else 0, code, _stream(index))
    if st != 0:
        raise FAError(st, "fa_rope")
    return q_out, k_out
