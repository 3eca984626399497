"""Timed cases of what a serving step does around attention over a paged cache, and a
training step around ``fa_fwd``: rotary positions and their gradient, the page tables and
slot maps of a step, and a KV cache held in 4 bits (writing, reading back, attention).

``run`` computes each operator in plain torch where ``own`` is false, and calls the
library's entry points where it is true.  Sizes: head counts, head dims and lengths are
those of the forward, decoding and 8-bit cache workloads of this repository.

The 4-bit cache is one byte tensor; for a page and head it holds, one after the other, the
codes of K [page, d / 2] (channel 2 c in the low half of byte c), the scales of K [page, d / 16],
and the same of V.  Scales and codes are defined without a choice, so that it is compared byte
for byte.
"""
import math
import random

import torch

own = False

DTYPES = {"fp16": torch.float16, "bf16": torch.bfloat16}
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
TOP_SCALE = 10240.0  # of a block, so that 6 of it fit fp16


def listed():
    return [
        # the query and key rows of one token at a decoding step: the call's latency
        dict(name="rope_step", op="rope", T=1, ctx=131072, Hq=32, Hkv=8, d=128, rot=128, interleaved=False,
             scaling="none", backward=False, dtype="bf16"),
        # ragged prompts of one step, rows of a fused projection, frequencies scaled for long contexts
        dict(name="rope_prompts", op="rope", T=58800, ctx=65536, Hq=32, Hkv=8, d=128, rot=128, interleaved=False,
             scaling="yarn", backward=False, dtype="bf16"),
        # the gradient in training, the base workload's shape, half of each head turned, neighbouring channels
        dict(name="rope_train", op="rope", B=4, N=2048, Hq=32, Hkv=32, d=64, rot=32, interleaved=True,
             scaling="none", backward=True, dtype="fp16"),
        # a speculative step of a serving batch: four tokens a sequence planned, some of them given back
        dict(name="pages_spec", op="spec", B=256, n=4, ctx=16384, page=16),
        # prompts admitted to a batch whose other sequences take one token each
        dict(name="pages_prompts", op="plan", B=64, n=16384, ctx=16384, page=64),
        # the decoding step of a full batch: one token of each sequence
        dict(name="write4_step", op="write4", B=256, n=1, ctx=16384, Hkv=8, d=128, page=16, dtype="bf16"),
        # ragged prompts written in one go, rows of a fused projection
        dict(name="write4_prompts", op="write4", B=6, n=16384, ctx=500, Hkv=8, d=128, page=64, dtype="fp16"),
        # one short prefix, small heads
        dict(name="read4_short", op="read4", B=1, len=1000, Hkv=32, d=64, page=32, dtype="fp16"),
        # cached prefixes of a batch read back for attention on 16-bit keys
        dict(name="read4_batch", op="read4", B=8, len=16384, Hkv=8, d=128, page=64, dtype="bf16"),
        # one short conversation: the smallest attention call
        dict(name="attend4_short", op="attend4", B=1, Nq=1, len=500, Hq=32, Hkv=8, d=128, page=64, dtype="bf16",
             causal=False),
        # four speculative tokens a sequence
        dict(name="attend4_spec", op="attend4", B=16, Nq=4, len=16384, Hq=32, Hkv=8, d=128, page=32, dtype="fp16",
             causal=True),
        # a serving batch of mixed lengths
        dict(name="attend4_batch", op="attend4", B=64, Nq=1, len=16384, Hq=32, Hkv=8, d=128, page=64, dtype="bf16",
             causal=False),
    ]


def _spread(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rope", "rope", "plan", "spec", "write4", "write4", "read4", "attend4", "attend4", "attend4"])
    d = rng.choice([32, 64, 96, 128, 128])
    Hkv = rng.choice([1, 2, 4, 8, 8, 32])
    dtype, page = rng.choice(["fp16", "bf16"]), rng.choice([16, 32, 64, 128])
    if op in ("plan", "spec"):
        B = _spread(rng, 1, 1024)
        n = _spread(rng, 1, min(16384, 500000 // B)) if op == "plan" else rng.randint(1, 8)
        return dict(op=op, B=B, n=n, ctx=_spread(rng, 16, 32768), page=page)
    if op == "rope":
        Hq = Hkv * rng.choice([1, 2, 4, 7, 8])
        if Hq > 128:
            Hq = Hkv
        case = dict(op=op, Hq=Hq, Hkv=Hkv, d=d, rot=rng.choice([d, d, d // 2, d // 4]), interleaved=rng.random() < 0.5,
                    scaling=rng.choice(["none", "linear", "base", "yarn"]), backward=rng.random() < 0.5, dtype=dtype)
        room = 55000 * 40 * 128 // ((Hq + Hkv) * d)
        if rng.random() < 0.3:
            N = _spread(rng, 1, min(16384, room))
            case.update(B=_spread(rng, 1, max(1, min(16, room // N))), N=N)
        else:
            case.update(T=_spread(rng, 1, min(100000, room)), ctx=_spread(rng, 1, 1000000))
        return case
    case = dict(op=op, Hkv=Hkv, d=d, page=page, dtype=dtype)
    # largest listed: 50,000 tokens of 8 heads of 128 (write), 70,000 (read), 64 x 8,700 (attend)
    if op == "write4":
        n = 1 if rng.random() < 0.5 else _spread(rng, 2, 16384)
        B = _spread(rng, 1, max(1, min(256, 45000 * 1024 // (n * Hkv * d))))
        case.update(B=B, n=n, ctx=_spread(rng, 1, 16384))
    elif op == "read4":
        length = _spread(rng, 1, 32768)
        case.update(B=_spread(rng, 1, max(1, min(64, 60000 * 1024 // (length * Hkv * d)))), len=length)
    else:
        G, Nq = rng.choice([1, 2, 4, 7, 8, 16]), rng.choice([1, 1, 1, 2, 3, 4])
        length = _spread(rng, 1, 131072)
        if Hkv * G > 128:
            G = 1
        B = _spread(rng, 1, max(1, min(128, 260000 * 1024 // (length * Hkv * d * max(1, Nq * G // 8)))))
        case.update(B=B, Nq=Nq, len=max(length, Nq), Hq=Hkv * G, causal=rng.random() < 0.5)
    return case


def _lengths(case):
    """Lengths of the batch's sequences: the same for every seed, the longest is the case's."""
    rng = random.Random("%s %s" % (case["B"], case["len"]))
    top = case["len"]
    return [top if b == 0 else max(case.get("Nq", 1), int(top * rng.uniform(0.05, 1.0))) for b in range(case["B"])]


def _writes(case):
    """(tokens before, new tokens) of each sequence."""
    rng = random.Random("%s %s %s" % (case["B"], case["n"], case["ctx"]))
    before, new = [], []
    for b in range(case["B"]):
        if case["op"] == "plan":  # every fourth a prompt, some with nothing to do
            before.append(rng.randrange(case["ctx"]) if b % 4 else 0)
            new.append(rng.choice([0, 1, 1, 1]) if b % 4 else max(1, int(case["n"] * rng.uniform(0.02, 1.0))))
        elif case["op"] == "spec" or case["n"] == 1:
            before.append(rng.randrange(case["ctx"]))
            new.append(case["n"])
        else:
            before.append(rng.randrange(case["ctx"]) if b % 2 else 0)
            new.append(case["n"] if b == 0 else max(1, int(case["n"] * rng.uniform(0.02, 0.9))))
    return before, new


def _padded(T):
    """Rows of a step's buffers, which a captured graph keeps: a few behind the last sequence."""
    return -(-T // 8) * 8


def _pages(n, page):
    return -(-n // page)


def _frequencies(case):
    """Radians a position of each pair, and the factor on turned channels."""
    rot, scaling = case["rot"], case["scaling"]
    base, stretch = 10000.0, 8.0
    if scaling == "base":
        base *= stretch ** (rot / max(2, rot - 2))
    w = [base ** (-2.0 * i / rot) for i in range(rot // 2)]
    if scaling == "linear":
        w = [x / stretch for x in w]
    if scaling == "yarn":  # pairs that turn seldom within the trained 8,192 positions are stretched, the others not
        at = [rot * math.log(8192 / (turns * 2 * math.pi)) / (2 * math.log(base)) for turns in (32.0, 1.0)]
        lo, hi = max(0, math.floor(at[0])), min(rot - 1, math.ceil(at[1]))
        part = [min(1.0, max(0.0, (i - lo) / max(hi - lo, 0.001))) for i in range(rot // 2)]
        return [x * (1 - y) + x / stretch * y for x, y in zip(w, part)], 0.1 * math.log(stretch) + 1.0
    return w, 1.0


# ---------------------------------------------------------------------------
# The plain forms


def _turn(x, cos, sin, rot, interleaved):
    """x [..., d] with its first rot channels turned; cos, sin broadcast to [..., rot / 2]."""
    y = x[..., :rot].float()
    a, b = (y[..., 0::2], y[..., 1::2]) if interleaved else (y[..., :rot // 2], y[..., rot // 2:])
    a, b = a * cos - b * sin, b * cos + a * sin
    y = torch.stack((a, b), -1).flatten(-2) if interleaved else torch.cat((a, b), -1)
    return torch.cat((y.to(x.dtype), x[..., rot:]), -1)


def _plain_rope(s):
    angle = s["positions"].double()[..., None] * s["radians"]
    cos, sin = (torch.cos(angle) * s["factor"]).float(), (torch.sin(angle) * s["factor"]).float()
    if s["backward"]:
        sin = -sin
    if s["q"].dim() == 3:
        cos, sin = cos[:, None], sin[:, None]
    return {name: _turn(s[name], cos, sin, s["rot"], s["interleaved"]) for name in ("q", "k")}


def _plain_plan(s):
    page, T, table, ring = s["page"], s["T"], s["table"], s["ring"].long()
    lens, n, counts = s["lens"].long(), s["n"].long(), s["counts"]
    cu = torch.cat((n.new_zeros(1), n.cumsum(0)))
    had = (lens + page - 1) // page
    fits = (lens + n <= table.shape[1] * page) & (cu[1:] <= T)
    need = torch.where(fits, (lens + n + page - 1) // page - had, 0)
    served = fits & ((need == 0) | (need.cumsum(0) <= counts[1] - counts[0]))
    need = torch.where(served, need, 0)
    # pages in the sequences' order, from the ring
    until = need.cumsum(0)
    j = torch.arange(T // page + len(lens) + 1, device=lens.device)
    seq = torch.searchsorted(until, j, right=True).clamp(max=len(lens) - 1)
    some = j < until[-1]
    at = had[seq] + j - (until - need)[seq]
    table[seq[some], at[some]] = ring[(counts[0] + j) % len(ring)][some].int()
    tok = torch.arange(T, device=lens.device)
    seq = torch.searchsorted(cu[1:], tok, right=True).clamp(max=len(lens) - 1)
    pos = torch.where((tok < cu[-1]) & served[seq], lens[seq] + tok - cu[seq], -1)
    slot = table[seq, (pos // page).clamp(min=0, max=table.shape[1] - 1)].long() * page + pos % page
    return {"table": table, "cu": cu.int(), "ends": torch.where(served, lens + n, lens).int(), "positions": pos.int(),
            "slots": torch.where(pos >= 0, slot, -1).int(), "counts": torch.stack((counts[0] + until[-1], counts[1]))}


def _plain_spec(s):
    out = _plain_plan(s)
    page, ring, counts = s["page"], s["ring"], out["counts"]
    keep = (s["keep"].long() + page - 1) // page
    back = (out["ends"].long() + page - 1) // page - keep
    until = back.cumsum(0)
    j = torch.arange(s["T"] // page + len(keep) + 1, device=keep.device)
    seq = torch.searchsorted(until, j, right=True).clamp(max=len(keep) - 1)
    some = j < until[-1]
    at = keep[seq] + j - (until - back)[seq]
    ring[((counts[1] + j) % len(ring))[some]] = s["table"][seq[some], at[some]]
    return {**out, "ring": ring, "counts": torch.stack((counts[0], counts[1] + until[-1]))}


def _block_scale(amax):
    """amax / 6 rounded to the nearest number of 5 exponent and 3 fraction bits, ties to even."""
    t = amax / 6.0
    step = (((torch.frexp(t).exponent.int().clamp(min=-13) - 4) + 127) << 23).view(torch.float32)  # exact, as pow() need not be
    return (torch.round(t / step) * step).clamp(max=TOP_SCALE)


def _encode(x):
    """Packed codes [..., d / 2] and scale bytes [..., d / 16] of fp32 x [..., d]."""
    x = x.unflatten(-1, (-1, 16))
    scale = _block_scale(x.abs().amax(-1))
    a = (x / scale[..., None]).abs()  # an IEEE quotient: exact where it is a tie
    code = ((a > 0.25).byte() + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5) + (a >= 3.5) + (a > 5)) | torch.signbit(x).byte() << 3
    code = torch.where(scale[..., None] > 0, code, 0).flatten(-2)
    return code[..., 0::2] | code[..., 1::2] << 4, (scale.half().view(torch.int16) >> 7).byte()


def _parts(data):
    """Views of K's codes and scales, and V's, of cache bytes [..., page, 9 d / 8]."""
    page, d = data.shape[-2], data.shape[-1] * 8 // 9
    x = data.flatten(-2)
    c, s = page * d // 2, page * d // 16
    return [x[..., at:at + n].unflatten(-1, (page, -1)) for at, n in ((0, c), (c, s), (c + s, c), (2 * c + s, s))]


def _decode(codes, scales):
    """fp32 values of packed codes [..., d / 2] and scale bytes [..., d / 16]."""
    value = torch.tensor(E2M1 + tuple(-x for x in E2M1), device=codes.device)
    x = value[torch.stack((codes & 15, codes >> 4), -1).flatten(-2).int()]
    scale = (scales.to(torch.int16) << 7).view(torch.float16).float()
    return (x.unflatten(-1, (-1, 16)) * scale[..., None]).flatten(-2)


def _plain_write4(s):
    page = s["page"]
    live = s["slots"] >= 0
    slots = s["slots"][live].long()
    parts = _parts(s["data"])
    for new, codes, scales in ((s["k_new"], *parts[:2]), (s["v_new"], *parts[2:])):
        c, e = _encode(new[live].float())
        codes[slots // page, :, slots % page] = c
        scales[slots // page, :, slots % page] = e
    return {"data": s["data"]}


def _gather(s):
    """fp32 K and V [B, Hkv, positions, d] of the sequences' pages."""
    parts = _parts(s["data"][s["table"].long()])
    return [_decode(c, e).transpose(1, 2).flatten(2, 3) for c, e in (parts[:2], parts[2:])]


def _plain_read4(s):
    live = (torch.arange(s["N"], device="cuda") < s["lens"][:, None])[:, None, :, None]
    k, v = (torch.where(live, x[:, :, :s["N"]], 0.0).to(s["dtype"]) for x in _gather(s))
    return {"k": k, "v": v}


def _plain_attend4(s):
    q = s["q"].float()
    B, Hq, Nq, d = q.shape
    k, v = _gather(s)
    G = Hq // k.shape[1]
    scores = (q.reshape(B, -1, G * Nq, d) @ k.transpose(-1, -2)) * d ** -0.5
    i = torch.arange(Nq, device=q.device)
    end = s["lens"][:, None].long() - ((Nq - 1 - i) if s["causal"] else 0 * i)  # keys that query i sees
    live = torch.arange(k.shape[2], device=q.device) < end.repeat(1, G)[..., None]
    scores = scores.masked_fill(~live[:, None], float("-inf"))
    m = scores.amax(-1, keepdim=True)
    p = torch.exp(scores - torch.where(torch.isinf(m), torch.zeros_like(m), m))
    total = p.sum(-1, keepdim=True)
    o = (p @ v) / torch.where(total > 0, total, torch.ones_like(total))
    return {"o": o.reshape(B, Hq, Nq, d).to(s["dtype"]), "lse": (torch.log(total) + m).reshape(B, Hq, Nq)}


PLAIN = {"rope": _plain_rope, "plan": _plain_plan, "spec": _plain_spec, "write4": _plain_write4, "read4": _plain_read4,
         "attend4": _plain_attend4}


# ---------------------------------------------------------------------------
# Inputs


def _values(shape, g):
    """Keys or values of pages [pages, Hkv, page, d]: a drift from page to page, a few strong channels, and noise."""
    pages, H, page, d = shape
    strong = 1.0 + 5.0 * (torch.rand(H, 1, d, generator=g, device="cuda") > 0.95)
    drift = torch.randn(pages, H, 1, d, generator=g, device="cuda") * 0.5
    return (torch.randn(shape, generator=g, device="cuda") + drift) * strong


def _filled(pages, case, g):
    """The bytes of `pages` pages of values."""
    H, page, d = case["Hkv"], case["page"], case["d"]
    data = torch.empty(pages, H, page, d * 9 // 8, dtype=torch.uint8, device="cuda")
    for at in range(0, pages, 4096):
        parts = _parts(data[at:at + 4096])
        for codes, scales in (parts[:2], parts[2:]):
            c, e = _encode(_values((min(4096, pages - at), H, page, d), g).to(DTYPES[case["dtype"]]).float())
            codes.copy_(c)
            scales.copy_(e)
    return data


def _prepare_rope(case, g):
    w, factor = _frequencies(case)
    s = {"rot": case["rot"], "interleaved": case["interleaved"], "backward": case["backward"], "factor": factor,
         "radians": torch.tensor(w, dtype=torch.float64, device="cuda"),
         # turns a position as fractions of 2^64, in two's complement
         "turns": torch.tensor([(int(x / (2 * math.pi) * 2.0 ** 64) + 2 ** 63) % 2 ** 64 - 2 ** 63 for x in w], device="cuda")}
    Hq, H, d, dtype = case["Hq"], case["Hkv"], case["d"], DTYPES[case["dtype"]]
    if "T" in case:
        # tokens of several sequences, each from a place of its own; rows as a fused projection gives them
        T = case["T"]
        cut = random.Random("%s %s" % (T, case["ctx"]))
        ends = sorted({T, *(cut.randrange(1, T + 1) for _ in range(min(7, T - 1)))})
        sizes = torch.tensor([e - b for b, e in zip([0, *ends], ends)], device="cuda")
        first = torch.randint(0, case["ctx"], (len(ends),), generator=g, device="cuda")
        begin = torch.repeat_interleave(first - torch.cumsum(sizes, 0) + sizes, sizes, output_size=T)
        s["positions"] = (begin + torch.arange(T, device="cuda")).int()
        x = torch.randn(T, Hq + 2 * H, d, generator=g, device="cuda").to(dtype)
        s["q"], s["k"] = x[:, :Hq], x[:, Hq:Hq + H]
    else:
        s["positions"] = torch.arange(case["N"], dtype=torch.int32, device="cuda")
        s["q"], s["k"] = (torch.randn(case["B"], h, case["N"], d, generator=g, device="cuda").to(dtype) for h in (Hq, H))
    return s


def _table(low, ends, g, spare=3):
    """A page table whose places low[b] .. ends[b] - 1 hold scattered pages, the others 0; and the pages of nobody."""
    need = sum(max(0, e - a) for a, e in zip(low, ends))
    order = torch.randperm(need + spare, generator=g, device="cuda").int()
    at = torch.tensor([0] + [max(0, e - a) for a, e in zip(low, ends)], device="cuda").cumsum(0)[:-1]
    col = torch.arange(max(1, *ends), device="cuda")
    lo, hi = (torch.tensor(x, device="cuda")[:, None] for x in (low, ends))
    index = (at[:, None] + col - lo).clamp(0, need + spare - 1)
    return torch.where((col >= lo) & (col < hi), order[index], 0), order[need:]


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed))
    op = case["op"]
    if op == "rope":
        return {"op": op, **_prepare_rope(case, g)}
    page, B = case["page"], case["B"]
    if op in ("plan", "spec"):
        before, new = _writes(case)
        had, ends = [_pages(b, page) for b in before], [_pages(b + n, page) for b, n in zip(before, new)]
        free = sum(ends) - sum(had) + 40
        table, rest = _table([0] * B, had, g, free)
        wide = torch.zeros(B, max(ends) + 1, dtype=torch.int32, device="cuda")
        wide[:, :min(table.shape[1], wide.shape[1])] = table[:, :wide.shape[1]]
        # the free pages lie in a ring of all pages, behind those taken and given back before
        pool = sum(had) + free
        taken = int(torch.randint(0, 10 * pool, (1,), generator=g, device="cuda"))
        ring = torch.full((pool,), -1, dtype=torch.int32, device="cuda")
        ring[(taken + torch.arange(free, device="cuda")) % pool] = rest
        s = {"op": op, "page": page, "T": _padded(sum(new)), "table": wide, "ring": ring,
             "lens": torch.tensor(before, dtype=torch.int32, device="cuda"), "n": torch.tensor(new, dtype=torch.int32, device="cuda"),
             "counts": torch.tensor([taken, taken + free], device="cuda"), "after": torch.zeros(2, dtype=torch.int64, device="cuda")}
        if op == "spec":
            kept = torch.randint(1, case["n"] + 1, (B,), generator=g, device="cuda")
            s["keep"] = (s["lens"] + kept).int()
        return s
    H, d, dtype = case["Hkv"], case["d"], DTYPES[case["dtype"]]
    s = {"op": op, "page": page, "dtype": dtype}
    if op == "write4":
        before, new = _writes(case)
        table, _ = _table([b // page for b in before], [_pages(b + n, page) for b, n in zip(before, new)], g)
        T = sum(new)
        s["data"] = _filled(sum(_pages(b + n, page) - b // page for b, n in zip(before, new)) + 3, case, g)
        sizes, start = (torch.tensor(x, device="cuda") for x in (new, before))
        seq = torch.repeat_interleave(torch.arange(B, device="cuda"), sizes, output_size=T)
        pos = start[seq] + torch.arange(T, device="cuda") - (sizes.cumsum(0) - sizes)[seq]
        s["slots"] = torch.full((_padded(T),), -1, dtype=torch.int32, device="cuda")
        s["slots"][:T] = (table[seq, pos // page] * page + pos % page).int()
        # key and value rows as a fused projection gives them: one buffer, [T, 2, Hkv, d]
        kv = torch.randn(_padded(T), 2, H, d, generator=g, device="cuda").to(dtype)
        s["k_new"], s["v_new"] = kv[:, 0], kv[:, 1]
        return s
    lens = _lengths(case)
    s["table"], _ = _table([0] * B, [_pages(n, page) for n in lens], g)
    s["data"] = _filled(sum(_pages(n, page) for n in lens) + 3, case, g)
    s["lens"] = torch.tensor(lens, dtype=torch.int32, device="cuda")
    if op == "read4":
        s["N"] = case["len"]
    else:
        s["causal"] = case["causal"]
        # query rows as a projection gives them, [B, Nq, Hq, d]
        s["q"] = torch.randn(B, case["Nq"], case["Hq"], d, generator=g, device="cuda").to(dtype).transpose(1, 2)
    return s


def run(s):
    if not own:
        return PLAIN[s["op"]](s)
    import attention_forward_02_gb300 as fa
    op = s["op"]
    if op == "rope":
        rope = fa.FARope(s["turns"], s["interleaved"], s["factor"])
        q, k = fa.fa_rope(s["q"], s["k"], rope, s["positions"], backward=s["backward"])
        return {"q": q, "k": k}
    if op in ("plan", "spec"):
        pool = fa.FAPagePool(s["ring"], s["counts"])
        plan = fa.fa_cache_plan(pool, s["table"], s["lens"], s["n"], s["page"], s["T"], counts=s["after"])
        out = {"table": s["table"], "cu": plan.cu_seqlens, "ends": plan.ends, "positions": plan.positions,
               "slots": plan.slots, "counts": s["after"]}
        if op == "spec":
            fa.fa_cache_trim(fa.FAPagePool(s["ring"], s["after"]), s["table"], plan.ends, s["keep"], s["page"])
            out["ring"] = s["ring"]
        return out
    cache = fa.FACache4(s["data"])
    if op == "write4":
        fa.fa_cache4_write(cache, s["k_new"], s["v_new"], s["slots"])
        return {"data": s["data"]}
    if op == "read4":
        k, v = fa.fa_cache4_read(cache, s["table"], s["lens"], s["N"], dtype=s["dtype"])
        return {"k": k, "v": v}
    o, lse = fa.fa_decode_cache4(s["q"], cache, s["table"], s["lens"], causal=s["causal"])
    return {"o": o, "lse": lse}


def work(case):
    op = case["op"]
    if op == "rope":
        rows = case["T"] if "T" in case else case["B"] * case["N"]
        at = case["T"] if "T" in case else case["N"]
        values = rows * (case["Hq"] + case["Hkv"])
        return {"bytes": values * case["d"] * 4 + 4 * at + 4 * case["rot"], "flops": values * case["rot"] * 3}
    if op in ("plan", "spec"):
        before, new = _writes(case)
        pages = sum(_pages(b + n, case["page"]) - _pages(b, case["page"]) for b, n in zip(before, new))
        more = 8 * case["B"] if op == "spec" else 0
        return {"bytes": 16 * case["B"] + 8 * _padded(sum(new)) + 8 * pages + more + 32, "flops": 0}
    H, d = case["Hkv"], case["d"]
    if op == "write4":
        T = sum(_writes(case)[1])
        return {"bytes": 2 * T * H * d * 2 + 2 * T * H * d * 9 // 16 + 4 * T, "flops": 2 * T * H * d * 2}
    lens = _lengths(case)
    codes = sum(lens) * H * d * 9 // 8
    table = 4 * sum(_pages(n, case["page"]) for n in lens)
    if op == "read4":
        return {"bytes": codes + table + 2 * case["B"] * case["len"] * H * d * 2, "flops": 2 * sum(lens) * H * d}
    rows = case["Hq"] * case["Nq"]
    return {"bytes": codes + table + case["B"] * rows * (4 * d + 4), "flops": 4 * rows * d * sum(lens)}


# ---------------------------------------------------------------------------
# The definitions in 64 bits, one sequence or token at a time


def _exact_rope(s, case):
    w, factor = _frequencies(case)
    angle = s["positions"].double()[:, None] * torch.tensor(w, dtype=torch.float64, device="cuda")
    by = torch.polar(torch.full_like(angle, factor), -angle if case["backward"] else angle)
    out = {}
    for name in ("q", "k"):
        x = s[name].double()
        half = case["rot"] // 2
        pairs = x[..., :case["rot"]].unflatten(-1, (half, 2) if case["interleaved"] else (2, half))
        pairs = pairs if case["interleaved"] else pairs.transpose(-1, -2)
        turned = torch.view_as_complex(pairs.contiguous()) * (by[:, None] if x.dim() == 3 else by)
        turned = torch.view_as_real(turned)
        turned = turned if case["interleaved"] else turned.transpose(-1, -2)
        x[..., :case["rot"]] = turned.flatten(-2)
        out[name] = x
    return out


def _exact_pages(s, case):
    page, ring, T = s["page"], s["ring"].tolist(), s["T"]
    lens, new, (taken, given) = s["lens"].tolist(), s["n"].tolist(), s["counts"].tolist()
    table = s["table"].tolist()
    cu, ends, positions, slots = [0], [], [], []
    for b, (had, n) in enumerate(zip(lens, new)):
        cu.append(cu[-1] + n)
        for at in range(_pages(had, page), _pages(had + n, page)):
            if taken == given:
                return None  # the pools here hold enough
            table[b][at] = ring[taken % len(ring)]
            taken += 1
        ends.append(had + n)
        for pos in range(had, had + n):
            positions.append(pos)
            slots.append(table[b][pos // page] * page + pos % page)
    out = {"table": table, "cu": cu, "ends": ends, "positions": positions + [-1] * (T - cu[-1]),
           "slots": slots + [-1] * (T - cu[-1])}
    if case["op"] == "spec":
        for b, keep in enumerate(s["keep"].tolist()):
            for at in range(_pages(keep, page), _pages(ends[b], page)):
                ring[given % len(ring)] = table[b][at]
                given += 1
        out["ring"] = ring
    out = {name: torch.tensor(x, dtype=torch.int32) for name, x in out.items()}
    return {**out, "counts": torch.tensor([taken, given])}


def _exact_encode(x):
    """Code numbers and scales of float64 x [..., d]: the nearest of all there are, ties to the even number."""
    x = x.unflatten(-1, (-1, 16))
    numbers = torch.arange(0, 0xE3, dtype=torch.int16, device=x.device)
    scales = (numbers << 7).view(torch.float16).double()
    at = _nearest(x.abs().amax(-1) / 6.0, scales)
    scale = scales[at]
    codes = _nearest(x.abs() / scale[..., None], torch.tensor(E2M1, dtype=torch.float64, device=x.device))
    codes = codes + 8 * torch.signbit(x).long()
    return torch.where(scale[..., None] > 0, codes, 0).flatten(-2), at


def _nearest(x, grid):
    """Number of the value of an ascending grid that is nearest to x, the even one at a tie."""
    hi = torch.searchsorted(grid, x.contiguous()).clamp(1, len(grid) - 1)
    lo = hi - 1
    up, down = grid[hi] - x, x - grid[lo]
    return torch.where((up < down) | ((up == down) & (hi % 2 == 0)), hi, lo)


def _exact_write4(s):
    page, data = s["page"], s["data"]
    P, H, _, wide = data.shape
    d = wide * 8 // 9
    data = data.reshape(P, H, -1)
    slots = s["slots"].long()
    where = torch.nonzero(slots >= 0)[:, 0]
    p, row = slots[where] // page, slots[where] % page
    h = torch.arange(H, device=data.device)[None, :, None]
    begin = 0
    for name in ("k_new", "v_new"):
        codes, scales = _exact_encode(s[name][where].double())
        both = codes[..., 0::2] + 16 * codes[..., 1::2]
        at = begin + row[:, None] * (d // 2) + torch.arange(d // 2, device=data.device)
        data[p[:, None, None], h, at[:, None]] = both.byte()
        at = begin + page * d // 2 + row[:, None] * (d // 16) + torch.arange(d // 16, device=data.device)
        data[p[:, None, None], h, at[:, None]] = scales.byte()
        begin += page * d // 2 + page * d // 16
    return {"data": data.reshape(s["data"].shape)}


def _exact_sequence(s, b, n):
    """float64 K and V [Hkv, positions, d] of the first n pages of sequence b."""
    blocks = s["data"][s["table"][b, :n].long()]
    page, d = blocks.shape[2], blocks.shape[3] * 8 // 9
    blocks = blocks.transpose(0, 1).flatten(2).long()
    out, at = [], 0
    for _ in range(2):
        codes = blocks[..., at:at + page * d // 2]
        at += page * d // 2
        scales = blocks[..., at:at + page * d // 16]
        at += page * d // 16
        code = torch.empty(*codes.shape[:-1], page * d, dtype=torch.int64, device=codes.device)
        code[..., 0::2], code[..., 1::2] = codes % 16, codes // 16
        sign, e, f = 1 - 2 * (code // 8), code // 2 % 4, code % 2
        value = sign * torch.where(e > 0, (2.0 + f) * 2.0 ** (e - 2).double(), 0.5 * f)
        se, sf = scales // 8, scales % 8
        scale = torch.where(se > 0, (8.0 + sf) * 2.0 ** (se - 18).double(), sf * 2.0 ** -17.0)
        out.append((value * scale.repeat_interleave(16, -1)).reshape(blocks.shape[0], -1, d))
    return out


def _exact_attend4(s, case):
    q = s["q"].double()
    B, Hq, Nq, d = q.shape
    o = torch.zeros(B, Hq, Nq, d, dtype=torch.float64, device=q.device)
    lse = torch.full((B, Hq, Nq), float("-inf"), dtype=torch.float64, device=q.device)
    for b, L in enumerate(s["lens"].tolist()):
        k, v = _exact_sequence(s, b, _pages(L, case["page"]))
        for i in range(Nq):
            end = L - (Nq - 1 - i) if case["causal"] else L
            if end < 1:
                continue
            x = torch.einsum("hgc,hjc->hgj", q[b, :, i].reshape(case["Hkv"], -1, d), k[:, :end]) / math.sqrt(d)
            z = torch.logsumexp(x, -1)
            o[b, :, i] = torch.einsum("hgj,hjc->hgc", torch.exp(x - z[..., None]), v[:, :end]).reshape(Hq, d)
            lse[b, :, i] = z.reshape(Hq)
    return {"o": o, "lse": lse}


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "rope":
        return _exact_rope(s, case)
    if case["op"] in ("plan", "spec"):
        return _exact_pages(s, case)
    if case["op"] == "write4":
        return _exact_write4(s)
    if case["op"] == "read4":
        out = {name: torch.zeros(case["B"], case["Hkv"], s["N"], case["d"], dtype=torch.float64, device="cuda") for name in "kv"}
        for b, L in enumerate(s["lens"].tolist()):
            k, v = _exact_sequence(s, b, _pages(L, case["page"]))
            out["k"][b, :, :L], out["v"][b, :, :L] = k[:, :L], v[:, :L]
        return out
    return _exact_attend4(s, case)
