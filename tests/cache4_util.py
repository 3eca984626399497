"""The 4-bit paged cache in 64 bits on the CPU, from the definition in include/fa.h, and the derived bounds that the
GPU tests hold the kernels to.  Writing and reading are compared for equality, attention with ``attend_bounds``."""
import math

import torch

DTYPES = {"fp16": torch.float16, "bf16": torch.bfloat16}
E2M1 = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], dtype=torch.float64)
# every scale byte's value: 5 exponent and 3 fraction bits, bias 15
SCALES = torch.tensor([(b & 7) * 2.0 ** -17 if b < 8 else (8 + (b & 7)) * 2.0 ** ((b >> 3) - 18) for b in range(0xE3)],
                      dtype=torch.float64)
AIM = 10    # log2 of a row's largest P in fp16, at least
STEP = 64   # keys of the smallest unit of work


def nearest(x, grid):
    """Number of the nearest value of an ascending grid, the even one at a tie."""
    hi = torch.searchsorted(grid, x.contiguous()).clamp(1, len(grid) - 1)
    up, down = grid[hi] - x, x - grid[hi - 1]
    return torch.where((up < down) | ((up == down) & (hi % 2 == 0)), hi, hi - 1)


def encode(x):
    """Code numbers [..., d] and scale bytes [..., d / 16] of 16-bit x."""
    x = x.double().unflatten(-1, (-1, 16))
    size = torch.where(torch.isfinite(x), x.abs(), 0.0)
    scale = nearest(size.amax(-1) / 6, SCALES)
    by = SCALES[scale][..., None]
    code = nearest((x.abs() / torch.where(by > 0, by, 1.0)).clamp(max=1e9).nan_to_num(0.0), E2M1) + 8 * torch.signbit(x).long()
    code = torch.where(torch.isnan(x) | (by == 0), 0, code)
    return code.flatten(-2), scale


def value(code, scale):
    """float64 values of code numbers and scale bytes (those that are no scales: NaN)."""
    by = torch.cat((SCALES, torch.full((256 - len(SCALES),), math.nan, dtype=torch.float64)))[scale.long()]
    code = code.long()
    x = E2M1[code & 7] * (1 - 2 * (code >> 3))
    return (x.unflatten(-1, (-1, 16)) * by[..., None]).flatten(-2)


class Ref:
    """A cache: code numbers k, v [num_pages, heads, page, d] and scale bytes."""

    def __init__(self, num_pages, heads, page, d, seed=0, lowest=0x50, highest=0x80):
        g = torch.Generator().manual_seed(seed)
        self.page, self.heads, self.d, self.num_pages = page, heads, d, num_pages
        shape = (num_pages, heads, page, d)
        self.k, self.v = (torch.randint(0, 16, shape, generator=g) for _ in range(2))
        self.k_scale, self.v_scale = (torch.randint(lowest, highest, (*shape[:3], d // 16), generator=g) for _ in range(2))

    def bytes(self):
        parts = []
        for code, scale in ((self.k, self.k_scale), (self.v, self.v_scale)):
            parts += [(code[..., 0::2] | code[..., 1::2] << 4).flatten(2), scale.flatten(2)]
        return torch.cat(parts, -1).to(torch.uint8).reshape(self.num_pages, self.heads, self.page, self.d // 8 * 9)

    def to(self, device):
        import attention_forward_02_gb300 as fa
        return fa.FACache4(self.bytes().to(device))

    def write(self, k, v, slots):
        for x, code, scale in ((k, self.k, self.k_scale), (v, self.v, self.v_scale)):
            c, s = encode(x)
            for t, slot in enumerate(slots):
                if 0 <= slot < self.num_pages * self.page:
                    code[slot // self.page, :, slot % self.page] = c[t]
                    scale[slot // self.page, :, slot % self.page] = s[t]

    def rows(self, table_row, n):
        """float64 k, v [heads, n, d] of a sequence's first n positions, and which of them have a page."""
        at = torch.arange(n)
        p = table_row[at // self.page].long() if n else at
        good = (p >= 0) & (p < self.num_pages)
        p = torch.where(good, p, 0)
        k = value(self.k[p, :, at % self.page], self.k_scale[p, :, at % self.page])
        v = value(self.v[p, :, at % self.page], self.v_scale[p, :, at % self.page])
        return k.transpose(0, 1), v.transpose(0, 1), good

    def read(self, table, lens, N, dtype):
        out = torch.zeros(2, len(lens), self.heads, N, self.d, dtype=torch.float64)
        for b, n in enumerate(lens):
            n = max(0, min(n, N, table.shape[1] * self.page))
            k, v, good = self.rows(table[b], n)
            out[0, b, :, :n] = torch.where(good[:, None], k, 0.0)
            out[1, b, :, :n] = torch.where(good[:, None], v, 0.0)
        return out.to(dtype)


def attend_bounds(ref, q, table, lens, scale, causal):
    """o and lse in 64 bits, and the bounds of |o - exact| and of |lse - exact|, from each row's own keys.

    With s_j a key's score, w_j its weight (they sum to one) over the n keys that the row sees:

    Scores.  K and Q are exact in fp16 (Q times a power of two), their products in fp32; the sum rounds or cuts
    each addition to 2^-23 of what it adds: d 2^-23 mag, mag the row's largest sum of magnitudes times scale.  Three fp32
    factors: 3 2^-24 mag.  The exponent s_j - m in log2 units, |m| <= top = 2 (mag / ln 2 + 16), is rounded with 2^-24 of
    each of its terms; the reference m moves by 4.9 at least each time but the first, (2 mag / ln 2) / 4.9 + 2 times, each with
    2^-24 top.  ex2.approx is good to 2^-22; merging warps and parts multiplies by two more such powers of two.
    Together, relative: r = (d + 8) 2^-23 mag + (moves + 8) 2^-24 top + 2^-20.

    The row sum adds n / 8 + 16 terms in a row at most (two of a 16-key tile a thread, then lanes and warps), and a
    merge of n / STEP + 1 parts: (n / 8 + n / STEP + 32) 2^-24.

    P is rounded to fp16: 2^-11 relative, or 2^-25 absolute below fp16's normal range, where 1 stands for 2^m and 2^m <=
    2^-AIM max_j w_j (1 + r) in units of the row sum.  V is exact in fp16.  The second product cuts each of a tile's 16
    terms and its sum so far at 2^-23 of the largest: 17/16 n 2^-23 of the sum of w_j |v_j|.  o is rounded once.
    """
    B, Hq, Nq, d = q.shape
    G = Hq // ref.heads
    fi = torch.finfo(q.dtype)
    o = torch.zeros(B, Hq, Nq, d, dtype=torch.float64)
    bo = torch.zeros_like(o)
    lse = torch.full((B, Hq, Nq), -math.inf, dtype=torch.float64)
    bl = torch.zeros(B, Hq, Nq, dtype=torch.float64)
    for b in range(B):
        n_all = max(0, min(lens[b], table.shape[1] * ref.page))
        k, v, good = ref.rows(table[b], n_all)
        for i in range(Nq):
            see = good & (torch.arange(n_all) < (n_all - Nq + 1 + i if causal else n_all))
            n = int(see.sum())
            if n == 0:
                continue
            x = q[b, :, i].double().unflatten(0, (ref.heads, G))
            kk, vv = k[:, see], v[:, see]
            s = torch.einsum("hgc,hjc->hgj", x, kk) * scale
            mag = torch.einsum("hgc,hjc->hgj", x.abs(), kk.abs()).amax(-1) * scale
            z = torch.logsumexp(s, -1)
            w = torch.exp(s - z[..., None])
            top = 2 * (mag / math.log(2) + 16)
            moves = 2 * mag / math.log(2) / 4.9 + 2
            r = (d + 8) * 2.0 ** -23 * mag + (moves + 8) * 2.0 ** -24 * top + 2.0 ** -20
            add = (n / 8 + n / STEP + 32) * 2.0 ** -24
            rel = 2 * r + 2 * add + 2.0 ** -11 + 17 / 16 * n * 2.0 ** -23
            want = torch.einsum("hgj,hjc->hgc", w, vv)
            a = torch.einsum("hgj,hjc->hgc", w, vv.abs())
            small = (w.amax(-1) * (1 + 2 * r))[..., None] * 2.0 ** (-25 - AIM) * vv.abs().sum(1)[:, None]
            off = fi.eps / 2 * want.abs() + (1 + fi.eps) * (rel[..., None] * a + small) + fi.tiny * fi.eps / 2
            o[b, :, i], bo[b, :, i] = want.flatten(0, 1), off.flatten(0, 1)
            lse[b, :, i] = z.flatten()
            bl[b, :, i] = (r + add + 2.0 ** -21 + 2.0 ** -22 * z.abs()).flatten()
    return o, lse, bo, bl


def within(o, lse, want):
    """Asserts that o and lse are within their bounds."""
    eo, el, bo, bl = want
    o, lse = o.cpu().double(), lse.cpu().double()
    empty = torch.isinf(el)
    assert torch.equal(torch.isneginf(lse), empty)
    assert (o[empty] == 0).all()
    over = ((o - eo).abs() / bo.clamp(min=1e-300))[~empty]
    assert over.numel() == 0 or over.max() <= 1, "o is off by %g of its bound" % over.max()
    over = ((lse - el).abs() / bl)[~empty]
    assert over.numel() == 0 or over.max() <= 1, "lse is off by %g of its bound" % over.max()


def pages_for(lens, page, seed, spare=2):
    """A page table with scattered pages (unused places hold the bad number -7) and the pool's size."""
    need = [-(-max(0, n) // page) for n in lens]
    pool = sum(need) + spare
    order = torch.randperm(pool, generator=torch.Generator().manual_seed(seed)).int()
    table = torch.full((len(lens), max(1, *need, 1) + 1), -7, dtype=torch.int32)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n]
        at += n
    return table, pool
