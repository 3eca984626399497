"""Rotary positions in 64 bits on the CPU, from the definition in include/fa.h, and the bound that the GPU tests
hold the kernel to."""
import math

import torch

DTYPES = {"fp16": torch.float16, "bf16": torch.bfloat16}


def turn(x, turns, interleaved, factor, positions, backward=False):
    """x [B, H, N, d] of any type as float64 y, and |a| + |b| of every channel's pair (0 where it stays).
    positions [B, N] of whole numbers (negative: the row stays)."""
    x = x.double()
    pairs = len(turns)
    y, mag = x.clone(), torch.zeros_like(x)
    first = [2 * i if interleaved else i for i in range(pairs)]
    second = [2 * i + 1 if interleaved else i + pairs for i in range(pairs)]
    angle = torch.zeros(*positions.shape, pairs, dtype=torch.float64)
    for b in range(positions.shape[0]):
        for n in range(positions.shape[1]):
            p = int(positions[b, n])
            angle[b, n] = torch.tensor([((int(t) * p) % 2 ** 64) / 2.0 ** 64 * 2 * math.pi for t in turns])
    cos, sin = torch.cos(angle)[:, None], torch.sin(angle)[:, None]
    if backward:
        sin = -sin
    stays = (positions < 0)[:, None, :, None]
    a, b = x[..., first], x[..., second]
    y[..., first] = torch.where(stays, a, factor * (a * cos - b * sin))
    y[..., second] = torch.where(stays, b, factor * (b * cos + a * sin))
    both = torch.where(stays, 0.0, (a.abs() + b.abs()) * abs(factor))
    mag[..., first], mag[..., second] = both, both
    return y, mag


def bound(y, mag, dtype):
    """Of |kernel - y|.  The angle is cut to 2^-32 of a turn and, in half turns below 1, rounded to fp32: off by
    2 pi 2^-32 + pi 2^-25 < 2^-23.  sincospif is good to 2 ulp of results up to 1, 2^-23; times the factor, rounded,
    2^-24 more.  Two products and their sum round with 2^-24 of the pair's magnitudes each, a fused one fewer.
    Together below 2^-21 of |a| + |b| times the factor.  Then one rounding to the type."""
    fi = torch.finfo(dtype)
    off = mag * 2.0 ** -21
    return fi.eps / 2 * (y.abs() + off) + off + fi.tiny * fi.eps / 2
