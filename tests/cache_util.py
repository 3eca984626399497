"""The 8-bit paged cache in 64 bits on the CPU, from the definition in
include/fa.h, and the derived bounds that the GPU tests hold the kernels to.

Writing, reading and page selection are exact but for one rounding each, so
they are compared for equality.  Attention is compared with ``bounds``.
"""
import math

import torch

DTYPES = {"fp16": torch.float16, "bf16": torch.bfloat16}
CODES = {"e4m3": torch.float8_e4m3fn, "int8": torch.int8}
TOP = {"e4m3": 448.0, "int8": 127.0}


def scale_of(amax, top):
    """Smallest 2^e, e >= -60, with amax <= top 2^e."""
    e = -60
    if amax > 0:
        e = max(e, math.frexp(amax / top)[1] - 1)
        while amax > top * 2.0 ** e:
            e += 1
    return 2.0 ** e


def encode(x, fmt):
    """Nearest code values (float64; int8: NaN becomes 0) of float64 x."""
    x = x.clamp(-TOP[fmt], TOP[fmt])
    if fmt == "int8":
        return torch.nan_to_num(x, nan=0.0).round()
    return x.float().to(torch.float8_e4m3fn).double()  # x is 16-bit times a power of two: float is exact


def as_codes(values, fmt):
    return values.float().to(CODES[fmt])


def finite_max(x):
    x = x.abs()
    x = x[x <= torch.finfo(torch.float64).max]
    return float(x.max()) if x.numel() else 0.0


class Ref:
    """A cache in float64: code values and scales."""

    def __init__(self, num_pages, heads, page, d, fmt, seed=0):
        g = torch.Generator().manual_seed(seed)
        self.page, self.fmt, self.heads, self.d = page, fmt, heads, d
        shape = (num_pages, heads, page, d)
        top = 100 if fmt == "int8" else 16
        self.k, self.v = (encode(torch.randn(shape, generator=g, dtype=torch.float64) * top, fmt) for _ in range(2))
        self.k_scale, self.v_scale = (2.0 ** torch.randint(-7, -3, shape[:2], generator=g).double() for _ in range(2))
        self.k_mean = torch.randint(-127, 128, (num_pages, heads, d), generator=g).double()
        self.k_mean_scale = 2.0 ** torch.randint(-8, -4, shape[:2], generator=g).double()

    def to(self, device, means=True):
        import attention_forward_02_gb300 as fa
        t = [as_codes(self.k, self.fmt), as_codes(self.v, self.fmt), self.k_scale.float(), self.v_scale.float()]
        if means:
            t += [self.k_mean.to(torch.int8), self.k_mean_scale.float()]
        return fa.FACache(*(x.to(device) for x in t))

    def summarise(self, p, h):
        codes = torch.nan_to_num(self.k[p, h], nan=0.0)
        mean = codes.sum(0) / self.page
        s = scale_of(float(mean.abs().max()), 127.0)
        self.k_mean[p, h] = (mean / s).round()
        self.k_mean_scale[p, h] = s * self.k_scale[p, h]

    def write(self, k, v, table, lens, cu):
        for b in range(len(lens)):
            t, end, pos = cu[b], cu[b + 1], lens[b]
            while t < end:
                slot, at = pos % self.page, pos // self.page
                n = min(self.page - slot, end - t)
                p = int(table[b, at]) if at < table.shape[1] else -1
                if 0 <= p < self.k.shape[0]:
                    for h in range(self.heads):
                        for x, codes, scale in ((k, self.k, self.k_scale), (v, self.v, self.v_scale)):
                            x = x[t:t + n, h].double()
                            s = scale_of(finite_max(x), TOP[self.fmt])
                            if slot:
                                s = max(s, float(scale[p, h]))
                                codes[p, h, :slot] = encode(codes[p, h, :slot] * (float(scale[p, h]) / s), self.fmt)
                            codes[p, h, slot:slot + n] = encode(x / s, self.fmt)
                            scale[p, h] = s
                        if slot + n == self.page:
                            self.summarise(p, h)
                t, pos = t + n, pos + n

    def sequence(self, table_row, n):
        """float64 k, v [heads, n, d] of a sequence's first n positions; a bad page's keys are NaN."""
        out = []
        for codes, scale in ((self.k, self.k_scale), (self.v, self.v_scale)):
            x = torch.full((self.heads, n, self.d), float("nan"), dtype=torch.float64)
            for at in range(-(-n // self.page)):
                p = int(table_row[at])
                m = min(self.page, n - at * self.page)
                if 0 <= p < self.k.shape[0]:
                    x[:, at * self.page:at * self.page + m] = codes[p, :, :m] * scale[p][:, None, None]
            out.append(x)
        return out

    def good(self, table_row, n):
        """Which of the first n positions lie in a page with a good number."""
        p = table_row[torch.arange(n) // self.page]
        return (p >= 0) & (p < self.k.shape[0])

    def select(self, q, table, lens, slots, first, last, causal):
        B, Hq, Nq, d = q.shape
        out = torch.full((B, self.heads, Nq, slots), -1, dtype=torch.int32)
        for b in range(B):
            for i in range(Nq):
                c = max(0, lens[b] - Nq + 1 + i if causal else lens[b])
                n = -(-c // self.page)
                for h in range(self.heads):
                    if n <= slots:
                        take = list(range(n))
                    else:
                        score = {}
                        for j in range(first, n - last):
                            p = int(table[b, j])
                            if not 0 <= p < self.k.shape[0]:
                                score[j] = -math.inf
                                continue
                            best = -math.inf
                            for g in range(Hq // self.heads):
                                x = q[b, h * (Hq // self.heads) + g, i].double()
                                s = scale_of(finite_max(x), 127.0)
                                x = encode(x / s, "int8")
                                best = max(best, float((x * self.k_mean[p, h]).sum()) * s * float(self.k_mean_scale[p, h]))
                            score[j] = best
                        take = sorted(score, key=lambda j: (-score[j], j))[:slots - first - last]
                        take = sorted(take + list(range(first)) + list(range(n - last, n)))
                    out[b, h, i, :len(take)] = torch.tensor(take, dtype=torch.int32)
        return out

    def attend(self, q, table, lens, scale, causal, pages=None):
        """o, lse and the terms of ``bounds``: sum of p |v|, and the largest sum of |q k| scale of a row."""
        B, Hq, Nq, d = q.shape
        G = Hq // self.heads
        o = torch.zeros(B, Hq, Nq, d, dtype=torch.float64)
        a = torch.zeros_like(o)
        lse = torch.full((B, Hq, Nq), -math.inf, dtype=torch.float64)
        mag = torch.zeros(B, Hq, Nq, dtype=torch.float64)
        for b in range(B):
            n = max(0, min(lens[b], table.shape[1] * self.page))
            if n == 0:
                continue
            k, v = self.sequence(table[b], n)
            ok = self.good(table[b], n)
            for hq in range(Hq):
                for i in range(Nq):
                    c = max(0, n - Nq + 1 + i if causal else n)
                    see = ok & (torch.arange(n) < c)
                    if pages is not None:
                        listed = torch.zeros(table.shape[1], dtype=torch.bool)
                        row = pages[b, hq // G, i][:-(-c // self.page)].long()
                        listed[row[row >= 0]] = True
                        see = see & listed[torch.arange(n) // self.page]
                    if not see.any():
                        continue
                    x = q[b, hq, i].double()
                    kk, vv = k[hq // G][see], v[hq // G][see]
                    s = (kk @ x) * scale
                    mag[b, hq, i] = (kk.abs() @ x.abs()).max() * scale
                    lse[b, hq, i] = torch.logsumexp(s, 0)
                    p = torch.exp(s - lse[b, hq, i])
                    o[b, hq, i], a[b, hq, i] = p @ vv, p @ vv.abs()
        return o, lse, a, mag


def bounds(ref, dtype, o, lse, a, mag, n, d):
    """Element-wise bounds of |o - exact| and |lse - exact|.

    A score is a sum of d products in fp32 (each partial sum rounded, or cut, to
    2^-23 of the sum of magnitudes at most) times three fp32 factors, and its
    exponential is ex2.approx, good to 2^-22: every weight p is off by at most
    r = (d + 8) 2^-23 mag + 2^-21 relative, which the row sum follows with as
    much again, plus n 2^-24 for n terms added in fp32.  Weights are rounded to
    fp16 for the second product: 2^-12 relative, or, below fp16's normal range,
    2^-25 of the largest possible weight times value (fp16 holds p times the V
    scale against a reference that is within 2 of the largest, so n 2^-24 of the
    largest value that the cache's V scales can stand for).  The second product
    adds n fp32 terms; o is rounded once to its type.
    """
    eps = torch.finfo(dtype).eps / 2
    r = (d + 8) * 2.0 ** -23 * mag + 2.0 ** -21
    top = TOP[ref.fmt] * float(ref.v_scale[torch.isfinite(ref.v_scale)].max())  # pages of nobody may hold NaN
    rel = 2 * r + 2.0 ** -12 + 2 * n * 2.0 ** -23
    bo = eps * o.abs() + (1 + eps) * (rel[..., None] * a + n * 2.0 ** -24 * top) + 2.0 ** -24
    bl = r + n * 2.0 ** -23 + 2.0 ** -22 * lse.abs() + 2.0 ** -22
    return bo, bl


def pages_for(lens, page, seed, spare=2):
    """A page table with scattered pages (unused places hold the bad number -7) and the pool's size."""
    need = [-(-max(0, n) // page) for n in lens]
    pool = sum(need) + spare
    order = torch.randperm(pool, generator=torch.Generator().manual_seed(seed)).int()
    table = torch.full((len(lens), max(1, *need) + 1 if len(need) > 1 else max(1, need[0]) + 1), -7, dtype=torch.int32)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n]
        at += n
    return table, pool
