"""Timed cases of the 8-bit paged KV cache: writing it, reading it back,
attending to it, and attending to the pages that a cheap score selects.

``run`` computes each operator in plain torch where ``own`` is false, and calls
the library's entry points where it is true.  Sizes: head counts and dims are
those of the decoding workloads (d = 128, up to 32 query heads, 16,384 to
131,072 keys) with grouped KV heads beside them.
"""
import math
import random

import torch

own = False

DTYPES = {"fp16": torch.float16, "bf16": torch.bfloat16}
CODES = {"e4m3": torch.float8_e4m3fn, "int8": torch.int8}
TOP = {"e4m3": 448.0, "int8": 127.0}
LOWEST = -60  # lowest scale exponent


def listed():
    return [
        # one token of one sequence appended at a decoding step: the call's latency
        dict(name="write_step_1", op="write", B=1, n=1, ctx=16384, Hkv=8, d=128, page=64, fmt="e4m3", dtype="bf16"),
        # the decoding step of a full batch, every sequence at its own place in its page
        dict(name="write_step_256", op="write", B=256, n=1, ctx=16384, Hkv=8, d=128, page=16, fmt="e4m3", dtype="bf16"),
        # ragged prompts written in one go, some after an earlier part of the prompt
        dict(name="write_prompts", op="write", B=6, n=16384, ctx=500, Hkv=8, d=128, page=64, fmt="int8", dtype="fp16"),
        # cached prefixes of a batch read back for attention on 16-bit keys
        dict(name="read_batch", op="read", B=8, len=16384, Hkv=8, d=128, page=64, fmt="e4m3", dtype="bf16"),
        # one short prefix, small heads
        dict(name="read_short", op="read", B=1, len=1000, Hkv=32, d=64, page=32, fmt="int8", dtype="fp16"),
        # one short conversation: the smallest attention call
        dict(name="attend_short", op="attend", B=1, Nq=1, len=500, Hq=32, Hkv=8, d=128, page=64, fmt="e4m3",
             dtype="bf16", causal=False),
        # one long document
        dict(name="attend_long", op="attend", B=1, Nq=1, len=131072, Hq=64, Hkv=8, d=128, page=64, fmt="e4m3",
             dtype="bf16", causal=False),
        # a serving batch of mixed lengths
        dict(name="attend_batch", op="attend", B=64, Nq=1, len=16384, Hq=32, Hkv=8, d=128, page=64, fmt="e4m3",
             dtype="bf16", causal=False),
        # four speculative tokens a sequence, int8 codes
        dict(name="attend_spec", op="attend", B=16, Nq=4, len=16384, Hq=32, Hkv=8, d=128, page=64, fmt="int8",
             dtype="fp16", causal=True),
        # as many KV heads as query heads, small heads and pages
        dict(name="attend_mha", op="attend", B=8, Nq=1, len=8000, Hq=32, Hkv=32, d=64, page=16, fmt="e4m3",
             dtype="fp16", causal=False),
        # sixty-four pages of a long document selected for its next token
        dict(name="sparse_long", op="sparse", B=1, Nq=1, len=131072, Hq=32, Hkv=8, d=128, page=64, slots=64,
             fmt="e4m3", dtype="bf16", causal=False),
        # a batch of long contexts, two tokens each
        dict(name="sparse_batch", op="sparse", B=32, Nq=2, len=65536, Hq=32, Hkv=4, d=128, page=32, slots=128,
             fmt="int8", dtype="bf16", causal=True),
    ]


def _spread(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["write", "read", "attend", "attend", "sparse", "sparse"])
    d = rng.choice([32, 64, 96, 128, 128])
    Hkv = rng.choice([1, 2, 4, 8, 8, 32])
    case = dict(op=op, Hkv=Hkv, d=d, page=rng.choice([16, 32, 64, 128]), fmt=rng.choice(["e4m3", "int8"]),
                dtype=rng.choice(["fp16", "bf16"]))
    # largest listed: about 64 x 8,700 tokens of 8 heads of 128 (attend), 50,000 tokens (write), 70,000 (read)
    if op == "write":
        n = 1 if rng.random() < 0.5 else _spread(rng, 2, 16384)
        B = _spread(rng, 1, max(1, min(256, 45000 * 1024 // (n * Hkv * d))))
        case.update(B=B, n=n, ctx=_spread(rng, 1, 16384))
    elif op == "read":
        length = _spread(rng, 1, 32768)
        B = _spread(rng, 1, max(1, min(64, 60000 * 1024 // (length * Hkv * d))))
        case.update(B=B, len=length)
    else:
        G = rng.choice([1, 2, 4, 7, 8, 16])
        Nq = rng.choice([1, 1, 1, 2, 3, 4])
        length = _spread(rng, 1 if op == "attend" else 600, 131072)
        if Hkv * G > 128:
            G = 1
        room = 260000 if op == "attend" else 500000
        B = _spread(rng, 1, max(1, min(128, room * 1024 // (length * Hkv * d * max(1, Nq * G // 8)))))
        case.update(B=B, Nq=Nq, len=max(length, Nq), Hq=Hkv * G, causal=rng.random() < 0.5)
        if op == "sparse":
            case["slots"] = max(3, _spread(rng, 256, 4096) // case["page"])
    return case


def _lengths(case):
    """Lengths of the batch's sequences: the same for every seed, the longest is the case's."""
    rng = random.Random("%s %s" % (case["B"], case.get("len", case.get("n"))))
    top = case["len"]
    return [top if b == 0 else max(case.get("Nq", 1), int(top * rng.uniform(0.05, 1.0))) for b in range(case["B"])]


def _writes(case):
    """(tokens before, tokens written) of each sequence."""
    rng = random.Random("%s %s %s" % (case["B"], case["n"], case["ctx"]))
    before, new = [], []
    for b in range(case["B"]):
        if case["n"] == 1:
            before.append(rng.randrange(case["ctx"]))
            new.append(1)
        else:
            before.append(rng.randrange(case["ctx"]) if b % 2 else 0)
            new.append(case["n"] if b == 0 else max(1, int(case["n"] * rng.uniform(0.02, 0.9))))
    return before, new


# ---------------------------------------------------------------------------
# The plain form


def _power(a, top):
    """2^e with the smallest e >= LOWEST such that a 2^-e <= top (a >= 0, finite)."""
    m, x = torch.frexp(a)
    tm, tx = math.frexp(top)
    e = torch.where(a > 0, x - tx + (m > tm).to(x.dtype), torch.full_like(x, LOWEST)).clamp(min=LOWEST)
    return ((e.int() + 127) << 23).view(torch.float32)  # exact, as pow() on the device need not be


def _finite_max(x, dim):
    return torch.where(torch.isfinite(x), x.abs(), torch.zeros_like(x)).amax(dim)


def _encode(x, fmt):
    """Nearest codes of fp32 values already divided by their scale, as bytes."""
    x = x.clamp(-TOP[fmt], TOP[fmt])
    if fmt == "e4m3":
        return x.to(torch.float8_e4m3fn).view(torch.uint8)
    return torch.nan_to_num(x, nan=0.0).round().to(torch.int8).view(torch.uint8)


def _decode(codes, fmt):
    """fp32 values of codes held as bytes."""
    return codes.view(CODES[fmt]).float()


def _summary(codes, scale, fmt):
    """int8 mean of the slots of whole pages [..., page, d] and its scale [...]."""
    mean = _decode(codes, fmt).double().mean(-2)
    p = _power(mean.abs().amax(-1).float(), 127.0)
    return (mean / p[..., None].double()).round().to(torch.int8), p * scale


def _plain_write(s):
    fmt, page = s["fmt"], s["page"]
    lens, cu, table = s["lens"].long(), s["cu"].long(), s["table"].long()
    n = cu[1:] - cu[:-1]
    T = s["k_new"].shape[0]
    tok = torch.arange(T, device=cu.device)
    seq = torch.searchsorted(cu, tok, right=True) - 1
    pos = lens[seq] + tok - cu[seq]
    first = lens // page
    J = (s["most"] + page - 2) // page + 1  # pages that a sequence can touch
    at = first[:, None] + torch.arange(J, device=cu.device)
    live = at * page < (lens + n)[:, None]
    pages = table.gather(1, at.clamp(max=table.shape[1] - 1))
    unit = seq * J + pos // page - first[seq]
    put = table[seq, pos // page]
    carry = ((lens % page > 0)[:, None] & (at == first[:, None]))[..., None]
    for new, codes, scale in ((s["k_new"], s["k"], s["k_scale"]), (s["v_new"], s["v"], s["v_scale"])):
        x = new.float()
        raw = codes.view(torch.uint8)
        top = torch.zeros(live.numel(), x.shape[1], device=x.device)
        top.scatter_reduce_(0, unit[:, None].expand(-1, x.shape[1]), _finite_max(x, -1), "amax")
        p = _power(top, TOP[fmt]).view(*live.shape, -1)
        old = scale[pages]
        p = torch.where(carry, torch.maximum(old, p), p)
        # the slots that a first page held before, at its new scale
        had = raw[pages[:, 0]]
        again = _encode(_decode(had, fmt) * (old[:, 0] / p[:, 0])[..., None, None], fmt)
        slot = torch.arange(page, device=cu.device)
        keep = (slot < (lens % page)[:, None]) & live[:, :1]
        some = live[:, 0]
        raw[pages[some, 0]] = torch.where(keep[:, None, :, None], again, had)[some]
        raw[put, :, pos % page] = _encode(x / p.view(-1, x.shape[1])[unit][..., None], fmt)
        scale[pages[live]] = p[live]
    done = pages[live & ((at + 1) * page <= (lens + n)[:, None])]
    s["k_mean"][done], s["k_mean_scale"][done] = _summary(s["k"].view(torch.uint8)[done], s["k_scale"][done], fmt)
    return {x: s[x] for x in ("k", "v", "k_scale", "v_scale", "k_mean", "k_mean_scale")}


def _gather(codes, scale, table, fmt):
    """[B, Hkv, positions, d] fp32 of the sequences' pages."""
    raw = _decode(codes.view(torch.uint8)[table], fmt) * scale[table][..., None, None]
    B, P, H, page, d = raw.shape
    return raw.permute(0, 2, 1, 3, 4).reshape(B, H, P * page, d)


def _plain_read(s):
    out = []
    for codes, scale in ((s["k"], s["k_scale"]), (s["v"], s["v_scale"])):
        x = _gather(codes, scale, s["table"].long(), s["fmt"])[:, :, :s["N"]]
        live = torch.arange(s["N"], device=x.device) < s["lens"][:, None]
        out.append(torch.where(live[:, None, :, None], x, torch.zeros_like(x)).to(s["dtype"]))
    return {"k": out[0], "v": out[1]}


def _attention(scores, live, v):
    """softmax over the live scores times v, and the log of its sum; nothing live: 0 and -inf."""
    scores = scores.masked_fill(~live, float("-inf"))
    m = scores.amax(-1, keepdim=True)
    p = torch.exp(scores - torch.where(torch.isinf(m), torch.zeros_like(m), m))
    total = p.sum(-1, keepdim=True)
    o = (p @ v) / torch.where(total > 0, total, torch.ones_like(total))
    return o, (torch.log(total) + m)[..., 0]


def _plain_attend(s):
    q = s["q"].float()
    B, Hq, Nq, d = q.shape
    Hkv = s["k"].shape[1]
    G = Hq // Hkv
    table = s["table"].long()
    k = _gather(s["k"], s["k_scale"], table, s["fmt"])
    v = _gather(s["v"], s["v_scale"], table, s["fmt"])
    scores = (q.reshape(B, Hkv, G * Nq, d) @ k.transpose(-1, -2)) * d ** -0.5
    i = torch.arange(Nq, device=q.device)
    end = s["lens"][:, None].long() - ((Nq - 1 - i) if s["causal"] else 0 * i)  # keys that query i sees
    live = torch.arange(k.shape[2], device=q.device) < end.repeat(1, G)[..., None]
    o, lse = _attention(scores, live[:, None], v)
    return {"o": o.reshape(B, Hq, Nq, d).to(s["dtype"]), "lse": lse.reshape(B, Hq, Nq)}


def _plain_sparse(s):
    q = s["q"].float()
    B, Hq, Nq, d = q.shape
    Hkv, page, S = s["k"].shape[1], s["page"], s["slots"]
    G = Hq // Hkv
    table = s["table"].long()
    P = table.shape[1]
    # scores of the pages: int8 query rows against int8 page means, exact in fp32
    qs = _power(_finite_max(q, -1), 127.0)
    q8 = torch.nan_to_num((q / qs[..., None]).clamp(-127, 127), nan=0.0).round()
    mean = s["k_mean"][table].float().permute(0, 2, 3, 1)
    by = s["k_mean_scale"][table].permute(0, 2, 1)
    dot = (q8.reshape(B, Hkv, G * Nq, d) @ mean).reshape(B, Hkv, G, Nq, P)
    score = ((dot * qs.reshape(B, Hkv, G, Nq, 1)) * by[:, :, None, None]).amax(2)
    i = torch.arange(Nq, device=q.device)
    end = s["lens"][:, None].long() - ((Nq - 1 - i) if s["causal"] else 0 * i)
    n = ((end + page - 1) // page)[:, None, :, None]
    j = torch.arange(P, device=q.device)
    score = torch.where((j < 1) | (j >= n - 1), torch.full_like(score, float("inf")), score)
    score = torch.where(j < n, score, torch.full_like(score, float("-inf")))
    best = torch.sort(score, dim=-1, descending=True, stable=True).indices[..., :S]
    best = torch.sort(torch.where(best < n, best, torch.full_like(best, P)), dim=-1).values
    if best.shape[-1] < S:
        best = torch.cat([best, best.new_full((*best.shape[:-1], S - best.shape[-1]), P)], -1)
    # attention over them
    phys = table.gather(1, best.clamp(max=P - 1).reshape(B, -1)).reshape(best.shape)
    h = torch.arange(Hkv, device=q.device)[:, None, None]
    kv = []
    for codes, scale in ((s["k"], s["k_scale"]), (s["v"], s["v_scale"])):
        x = _decode(codes.view(torch.uint8)[phys, h], s["fmt"]) * scale[phys, h][..., None, None]
        kv.append(x.reshape(B, Hkv, Nq, S * page, d))
    rows = q.reshape(B, Hkv, G, Nq, d).transpose(2, 3)
    scores = (rows @ kv[0].transpose(-1, -2)) * d ** -0.5
    pos = (best[..., None] * page + torch.arange(page, device=q.device)).reshape(B, Hkv, Nq, 1, S * page)
    o, lse = _attention(scores, (pos < end[:, None, :, None, None]) & (pos < P * page), kv[1])
    return {"pages": torch.where(best < P, best, torch.full_like(best, -1)).int(),
            "o": o.transpose(2, 3).reshape(B, Hq, Nq, d).to(s["dtype"]), "lse": lse.transpose(2, 3).reshape(B, Hq, Nq)}


# ---------------------------------------------------------------------------
# Inputs


def _values(shape, g, dtype):
    """Keys or values of pages [pages, Hkv, page, d]: a drift from page to page, a few strong channels, and noise."""
    pages, H, page, d = shape
    strong = 1.0 + 5.0 * (torch.rand(H, 1, d, generator=g, device="cuda") > 0.95)
    drift = torch.randn(pages, H, 1, d, generator=g, device="cuda") * 0.5
    return ((torch.randn(shape, generator=g, device="cuda") + drift) * strong).to(dtype)


def _filled(pages, case, g):
    """Codes and scales of `pages` pages of values."""
    got, H, page, d = {}, case["Hkv"], case["page"], case["d"]
    for name in ("k", "v"):
        codes = torch.empty(pages, H, page, d, dtype=torch.uint8, device="cuda")
        scale = torch.empty(pages, H, device="cuda")
        for at in range(0, pages, 4096):
            x = _values((min(4096, pages - at), H, page, d), g, DTYPES[case["dtype"]]).float()
            p = _power(_finite_max(x, -1).amax(-1), TOP[case["fmt"]])
            codes[at:at + 4096] = _encode(x / p[..., None, None], case["fmt"])
            scale[at:at + 4096] = p
        got[name], got[name + "_scale"] = codes.view(CODES[case["fmt"]]), scale
    got["k_mean"] = torch.empty(pages, H, d, dtype=torch.int8, device="cuda")
    got["k_mean_scale"] = torch.empty(pages, H, device="cuda")
    for at in range(0, pages, 4096):
        m, p = _summary(got["k"].view(torch.uint8)[at:at + 4096], got["k_scale"][at:at + 4096], case["fmt"])
        got["k_mean"][at:at + 4096], got["k_mean_scale"][at:at + 4096] = m, p
    return got


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed))
    H, d, page, dtype = case["Hkv"], case["d"], case["page"], DTYPES[case["dtype"]]
    s = {"op": case["op"], "fmt": case["fmt"], "page": page, "dtype": dtype}
    if case["op"] == "write":
        before, new = _writes(case)
        low = [b // page for b in before]  # pages below are not touched: their places in the table stay 0
        ends = [-(-(b + n) // page) for b, n in zip(before, new)]
    else:
        before = _lengths(case)
        low, ends = [0] * len(before), [-(-b // page) for b in before]
    need = sum(e - a for a, e in zip(low, ends))
    pool = need + 3
    order = torch.randperm(pool, generator=g, device="cuda").int()
    at = torch.tensor([0] + [e - a for a, e in zip(low, ends)], device="cuda").cumsum(0)[:-1]
    col = torch.arange(max(ends), device="cuda")
    lo, hi = (torch.tensor(x, device="cuda")[:, None] for x in (low, ends))
    index = (at[:, None] + col - lo).clamp(0, pool - 1)
    s["table"] = torch.where((col >= lo) & (col < hi), order[index], torch.zeros_like(order[index]))
    s["lens"] = torch.tensor(before, dtype=torch.int32, device="cuda")
    s.update(_filled(pool, case, g))
    if case["op"] == "write":
        cu = [0]
        for n in new:
            cu.append(cu[-1] + n)
        s["cu"] = torch.tensor(cu, dtype=torch.int32, device="cuda")
        s["most"] = max(new)
        # key and value rows as a fused projection gives them: one buffer, [T, 2, Hkv, d]
        kv = torch.randn(cu[-1], 2, H, d, generator=g, device="cuda").to(dtype)
        s["k_new"], s["v_new"] = kv[:, 0], kv[:, 1]
    elif case["op"] == "read":
        s["N"] = case["len"]
    else:
        s["causal"], s["slots"] = case["causal"], case.get("slots", 0)
        # query rows as a projection gives them, [B, Nq, Hq, d]
        q = torch.randn(case["B"], case["Nq"], case["Hq"], d, generator=g, device="cuda").to(dtype)
        s["q"] = q.transpose(1, 2)
    return s


def run(s):
    if not own:
        return {"write": _plain_write, "read": _plain_read, "attend": _plain_attend, "sparse": _plain_sparse}[s["op"]](s)
    import attention_forward_02_gb300 as fa
    cache = fa.FACache(s["k"], s["v"], s["k_scale"], s["v_scale"], s["k_mean"], s["k_mean_scale"])
    if s["op"] == "write":
        fa.fa_cache_write(cache, s["k_new"], s["v_new"], s["table"], s["lens"], cu_seqlens=s["cu"])
        return cache._asdict()
    if s["op"] == "read":
        k, v = fa.fa_cache_read(cache, s["table"], s["lens"], s["N"], dtype=s["dtype"])
        return {"k": k, "v": v}
    if s["op"] == "attend":
        o, lse = fa.fa_decode_cache(s["q"], cache, s["table"], s["lens"], causal=s["causal"])
        return {"o": o, "lse": lse}
    pages = fa.fa_cache_select(s["q"], cache, s["table"], s["lens"], s["slots"], causal=s["causal"])
    o, lse = fa.fa_decode_cache(s["q"], cache, s["table"], s["lens"], pages=pages, causal=s["causal"])
    return {"pages": pages, "o": o, "lse": lse}


def work(case):
    H, d, page = case["Hkv"], case["d"], case["page"]
    if case["op"] == "write":
        before, new = _writes(case)
        T = sum(new)
        pages = sum(-(-(b + n) // page) - b // page for b, n in zip(before, new))
        return {"bytes": 2 * T * H * d * 3 + 8 * pages * H, "flops": 2 * T * H * d * 3}
    lens = _lengths(case)
    if case["op"] == "read":
        return {"bytes": 2 * sum(lens) * H * d + 2 * case["B"] * case["len"] * H * d * 2, "flops": 2 * sum(lens) * H * d}
    rows = case["Hq"] * case["Nq"]
    small = case["B"] * rows * (4 * d + 4) + 4 * sum(-(-x // page) for x in lens)
    if case["op"] == "attend":
        return {"bytes": sum(lens) * H * 2 * d + sum(-(-x // page) for x in lens) * H * 8 + small,
                "flops": 4 * rows * d * sum(lens)}
    pages = [-(-x // page) for x in lens]
    keys = sum(min(x, case["slots"] * page) for x in lens)
    # the pages of one query of each sequence at least, whatever its other queries select
    return {"bytes": sum(pages) * H * (d + 4) + keys * H * 2 * d + 4 * case["B"] * H * case["Nq"] * case["slots"] + small,
            "flops": 2 * rows * d * sum(pages) + 4 * rows * d * keys}


# ---------------------------------------------------------------------------
# The definition in 64 bits, one sequence (and page) at a time


def _two(e):
    """2^e in float64, exactly, for a tensor of whole numbers."""
    return ((e.long() + 1023) << 52).view(torch.float64)


def _exact_scale(a, top):
    """Smallest 2^e, e >= LOWEST, with a <= top 2^e, for a float64 tensor a >= 0."""
    e = torch.ceil(torch.log2(a.clamp(min=1e-300) / top))
    e = torch.where(a > top * _two(e), e + 1, e)
    e = torch.where(a <= top * _two(e - 1), e - 1, e)
    return _two(e.clamp(min=LOWEST))


def _nearest(x, fmt):
    x = x.clamp(-TOP[fmt], TOP[fmt])
    if fmt == "int8":
        return torch.round(x)
    step = _two((torch.frexp(x).exponent - 1).clamp(min=-6) - 3)
    return torch.round(x / step) * step


def _exact_write(s):
    fmt, page, out = s["fmt"], s["page"], {}
    lens, cu, table = s["lens"].tolist(), s["cu"].tolist(), s["table"].tolist()
    units = []  # (page, first new slot, first token, tokens)
    for b, L in enumerate(lens):
        t, end = cu[b], cu[b + 1]
        while t < end:
            pos = L + t - cu[b]
            count = min(page - pos % page, end - t)
            units.append((table[b][pos // page], pos % page, t, count))
            t += count
    for name in ("k", "v"):
        new, codes = s[name + "_new"].double(), s[name].view(torch.uint8).view(CODES[fmt]).double()
        scale = s[name + "_scale"].double()
        for p, slot, t, count in units:
            x = new[t:t + count].transpose(0, 1)
            e = _exact_scale(x.abs().amax((1, 2)), TOP[fmt])
            if slot:
                e = torch.maximum(e, scale[p])
                codes[p, :, :slot] = _nearest(codes[p, :, :slot] * (scale[p] / e)[:, None, None], fmt)
            codes[p, :, slot:slot + count] = _nearest(x / e[:, None, None], fmt)
            scale[p] = e
        out[name], out[name + "_scale"] = codes, scale
    mean, by = s["k_mean"].double(), s["k_mean_scale"].double()
    for p, slot, t, count in units:
        if slot + count == page:
            m = out["k"][p].sum(1) / page
            e = _exact_scale(m.abs().amax(1), 127.0)
            mean[p], by[p] = torch.round(m / e[:, None]), e * out["k_scale"][p]
    return {**out, "k_mean": mean.to(torch.int8), "k_mean_scale": by}


def _sequence(s, name, b, n):
    """[Hkv, n pages * page, d] float64 of the first n pages of sequence b."""
    at = s["table"][b, :n].long()
    x = s[name].view(torch.uint8)[at].view(CODES[s["fmt"]]).double() * s[name + "_scale"][at].double()[..., None, None]
    return x.transpose(0, 1).reshape(x.shape[1], -1, x.shape[3])


def _exact_attend(s, case, chosen=None):
    q = s["q"].double()
    B, Hq, Nq, d = q.shape
    G = Hq // case["Hkv"]
    o = torch.zeros(B, Hq, Nq, d, dtype=torch.float64, device=q.device)
    lse = torch.full((B, Hq, Nq), float("-inf"), dtype=torch.float64, device=q.device)
    for b, L in enumerate(s["lens"].tolist()):
        k, v = (_sequence(s, name, b, -(-L // case["page"])) for name in ("k", "v"))
        for i in range(Nq):
            end = L - (Nq - 1 - i) if case["causal"] else L
            if end < 1:
                continue
            x = torch.einsum("hgc,hjc->hgj", q[b, :, i].reshape(-1, G, d), k[:, :end]) / math.sqrt(d)
            if chosen is not None:
                keep = chosen[b, :, i][:, torch.arange(end, device=q.device) // case["page"]]
                x = x.masked_fill(~keep[:, None], float("-inf"))
            z = torch.logsumexp(x, -1)
            o[b, :, i] = torch.einsum("hgj,hjc->hgc", torch.exp(x - z[..., None]), v[:, :end]).reshape(Hq, d)
            lse[b, :, i] = z.reshape(Hq)
    return {"o": o, "lse": lse}


def _exact_sparse(s, case):
    q = s["q"].double()
    B, Hq, Nq, d = q.shape
    Hkv, S, page = case["Hkv"], case["slots"], case["page"]
    P = s["table"].shape[1]
    pages = torch.full((B, Hkv, Nq, S), -1, dtype=torch.int32)
    chosen = torch.zeros(B, Hkv, Nq, P, dtype=torch.bool, device=q.device)
    for b, L in enumerate(s["lens"].tolist()):
        at = s["table"][b].long()
        for i in range(Nq):
            n = -(-(L - (Nq - 1 - i) if case["causal"] else L) // page)
            if n <= S:
                take = [list(range(n))] * Hkv
            else:
                rows = q[b, :, i]
                e = _exact_scale(rows.abs().amax(-1), 127.0)
                rows = torch.round(rows / e[:, None]) * e[:, None]
                x = torch.einsum("hgc,jhc->hgj", rows.reshape(Hkv, -1, d), s["k_mean"][at[:n]].double())
                x = (x * s["k_mean_scale"][at[:n]].double().t()[:, None]).amax(1)[:, 1:n - 1]
                best = torch.argsort(-x, dim=-1, stable=True)[:, :S - 2] + 1
                take = [sorted([0, n - 1] + row) for row in best.tolist()]
            for h, row in enumerate(take):
                pages[b, h, i, :len(row)] = torch.tensor(row, dtype=torch.int32)
                chosen[b, h, i, row] = True
    return {"pages": pages, **_exact_attend(s, case, chosen)}


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "write":
        return _exact_write(s)
    if case["op"] == "read":
        out = {}
        for name in ("k", "v"):
            x = torch.zeros(case["B"], case["Hkv"], s["N"], case["d"], dtype=torch.float64, device="cuda")
            for b, L in enumerate(s["lens"].tolist()):
                x[b, :, :L] = _sequence(s, name, b, -(-L // case["page"]))[:, :L]
            out[name] = x
        return out
    if case["op"] == "attend":
        return _exact_attend(s, case)
    return _exact_sparse(s, case)
