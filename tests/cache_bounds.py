"""Bounds of attention over the 8-bit cache, row by row.

Each row's bound comes from the keys, weights and V codes of that row alone, so
a value of V that is lost, doubled or taken from another place shows even where
thousands of keys share the weight.
"""
import math

import torch

from cache_util import TOP

# The kernel's softmax reference lies so that a row's largest P * v_scale (its
# power of two) is at least 2^AIM in fp16.
AIM = 10
STEP = 64  # keys of the smallest unit of work


def attend_bounds(ref, q, table, lens, scale, causal, pages=None):
    """o and lse in 64 bits, and the bounds of |o - exact| and of |lse - exact|.

    With s_j a key's score, w_j its weight (they sum to one), c_j its V code and
    2^v_j r_j its V scale (1 <= r_j < 2), over the n keys that the row sees:

    Scores.  The product of a row with a key adds d exact products in fp32, each
    addition rounded or cut to 2^-23 of what it adds: d 2^-23 mag, mag the largest
    sum of magnitudes of a row, times scale.  Three fp32 factors: 3 2^-24 mag.  The
    exponent s_j + v_j - m in log2 units, |m| <= top = 2 (mag / ln 2 + largest |v_j| + 16),
    is rounded with 2^-24 of each of its terms; the reference m moves at most once per
    unit of growth, 2 (mag / ln 2 + spread of v_j) + 1 times, each with 2^-24 top.
    ex2.approx is good to 2^-22.  Merging warps and parts multiplies by two more such
    powers of two.  Together, relative: r = (d + 8) 2^-23 mag + (moves + 8) 2^-24 top + 2^-20.

    The row sum adds n / 8 + 16 terms in a row at most (two of a 16-key tile a thread,
    then lanes and warps), and a merge of n / STEP + 1 parts: (n / 8 + n / STEP + 32) 2^-24.

    P * v_scale is rounded to fp16: 2^-12 relative (2^-24 more for the factor r_j), or
    2^-25 absolute below fp16's normal range, where 1 stands for 2^m, and
    2^m <= 2^-AIM max_j(w_j 2^v_j) (1 + r) in units of the row sum.
    The second product cuts each of a tile's 16 terms and its sum so far at 2^-23 of the
    largest: 17/16 n 2^-23 of the sum of w_j |V_j|, merges (n / STEP + 32) 2^-24.
    o is rounded once to its type.
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
        if n_all == 0:
            continue
        at = torch.arange(n_all)
        page = table[b, at // ref.page].long()
        ok = ref.good(table[b], n_all)
        page = torch.where(ok, page, torch.zeros_like(page))
        slot = at % ref.page
        for hq in range(Hq):
            h = hq // G
            kc, vc = ref.k[page, h, slot], ref.v[page, h, slot]
            ks, vs = ref.k_scale[page, h], ref.v_scale[page, h]
            for i in range(Nq):
                see = ok & (at < (n_all - Nq + 1 + i if causal else n_all))
                if pages is not None:
                    c = max(0, n_all - Nq + 1 + i if causal else n_all)
                    listed = torch.zeros(table.shape[1], dtype=torch.bool)
                    row = pages[b, h, i][:-(-c // ref.page)].long()
                    listed[row[row >= 0]] = True
                    see = see & listed[at // ref.page]
                n = int(see.sum())
                if n == 0:
                    continue
                x = q[b, hq, i].double()
                kk, code, vscale = kc[see] * ks[see][:, None], vc[see], vs[see]
                s = (kk @ x) * scale
                mag = float((kk.abs() @ x.abs()).max()) * scale
                z = torch.logsumexp(s, 0)
                w = torch.exp(s - z)
                v = code * vscale[:, None]
                two = torch.floor(torch.log2(vscale))
                top = 2 * (mag / math.log(2) + float(two.abs().max()) + 16)
                moves = 2 * (mag / math.log(2) + float(two.max() - two.min())) + 1
                r = (d + 8) * 2.0 ** -23 * mag + (moves + 8) * 2.0 ** -24 * top + 2.0 ** -20
                add = (n / 8 + n / STEP + 32) * 2.0 ** -24
                a = w @ v.abs()
                small = float((w * 2.0 ** two).max()) * (1 + 2 * r) * 2.0 ** (-25 - AIM) * code.abs().sum(0)
                rel = 2 * r + 2 * add + 2.0 ** -12 + 2.0 ** -23 + 17 / 16 * n * 2.0 ** -23
                o[b, hq, i], lse[b, hq, i] = w @ v, z
                bo[b, hq, i] = (fi.eps / 2 * o[b, hq, i].abs() + (1 + fi.eps) * (rel * a + small)
                                + fi.tiny * fi.eps / 2)
                bl[b, hq, i] = r + add + 2.0 ** -21 + 2.0 ** -22 * abs(float(z))
    return o, lse, bo, bl


def excess(o, lse, want):
    """How far o and lse are over their bounds at the worst element (<= 0: within), in units of the bound."""
    eo, el, bo, bl = want
    some = ~torch.isinf(el)
    over = ((o - eo).abs() / bo)[some].max() - 1 if some.any() else torch.tensor(0.0)
    lse_over = ((lse - el).abs() / bl)[some].max() - 1 if some.any() else torch.tensor(0.0)
    return float(over), float(lse_over)


def tiles_apart(ref, seed=5):
    """Values whose sign is each tile's of 16 keys, head's and channel's, so that a tile's share of o adds up."""
    g = torch.Generator().manual_seed(seed)
    P, H, page, d = ref.v.shape
    sign = torch.randint(0, 2, (P, H, page // 16, 1, d), generator=g).double() * 2 - 1
    ref.v = (ref.v.abs().reshape(P, H, page // 16, 16, d) * sign).reshape(ref.v.shape)
    return ref


def sink(ref, table, lens, q, at, mass):
    """Key `at` of each sequence (head 0 ..) with V = 0 that takes about `mass` of each first row's weight: the key
    is the query's direction, q is made the same for all rows of a KV head, and its score found by bisection."""
    B, Hq, Nq, d = q.shape
    G = Hq // ref.heads
    for b in range(B):
        p, slot = int(table[b, at // ref.page]), at % ref.page
        for h in range(ref.heads):
            x = torch.sign(torch.randn(d, generator=torch.Generator().manual_seed(7 * b + h)))
            q[b, h * G:(h + 1) * G] = x.to(q.dtype)
            ref.v[p, h, slot] = 0.0
            k, _ = ref.sequence(table[b], lens[b])
            s = (k[h] @ x.double()) * d ** -0.5
            s[at] = -math.inf
            want = float(torch.logsumexp(s, 0)) + math.log(mass / (1 - mass))
            # a code a channel, as many as reach the score: s = scale * k_scale * sum of codes
            left = round(want * d ** 0.5 / float(ref.k_scale[p, h]))
            codes = torch.zeros(d, dtype=torch.float64)
            for c in range(d):
                step = min(left, 120)
                if ref.fmt == "e4m3" and step > 16:  # four bits
                    step = step // 2 * 2 if step < 32 else step // 4 * 4 if step < 64 else step // 8 * 8
                codes[c] = step
                left -= step
            ref.k[p, h, slot] = codes * x.double()
