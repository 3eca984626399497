"""The 4-bit paged cache on the GPU: writing and reading equal to the definition, attention within derived bounds."""
import math

import pytest
import torch

import attention_forward_02_gb300 as fa
from cache4_util import DTYPES, Ref, attend_bounds, pages_for, within

pytestmark = pytest.mark.gpu
DEV = "cuda"


def normal(shape, dtype, seed, by=1.0):
    return (torch.randn(shape, generator=torch.Generator().manual_seed(seed)) * by).to(DTYPES[dtype])


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def status():
    return fa.fa_last_device_status(torch.cuda.current_stream().cuda_stream)


def same(cache, ref):
    assert torch.equal(cache.data.cpu(), ref.bytes())


# ---------------------------------------------------------------------------
# writing


def bits(shape, dtype, seed):
    """Any 16-bit patterns: every exponent, infinities and NaN among them."""
    x = torch.randint(-2 ** 15, 2 ** 15, shape, generator=torch.Generator().manual_seed(seed)).to(torch.int16)
    return x.view(DTYPES[dtype])


def close(shape, dtype, seed):
    """Values of one block near one another, many on the borders between codes."""
    g = torch.Generator().manual_seed(seed)
    step = torch.randint(0, 49, shape, generator=g) / 8.0        # multiples of an eighth up to 6
    sign = torch.randint(0, 2, shape, generator=g) * 2 - 1
    block = torch.randint(8, 16, (*shape[:-1], shape[-1] // 16, 1), generator=g) * 2.0 ** torch.randint(
        -16, 10 if dtype == "fp16" else 11, (*shape[:-1], shape[-1] // 16, 1), generator=g).float()
    x = (step.unflatten(-1, (-1, 16)) * block).flatten(-2) * sign
    x = x.clamp(-65504, 65504).to(DTYPES[dtype])
    nudge = torch.randint(-1, 2, shape, generator=g).to(torch.int16)
    return (x.view(torch.int16) + torch.where(x == 0, 0, nudge)).view(DTYPES[dtype])


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("d", [32, 64, 96, 128])
@pytest.mark.parametrize("page", [16, 32, 64, 128])
def test_write(dtype, d, page):
    """Scattered slots, padding, rows of a fused projection; nothing else changes."""
    H, P, T = 3, 5, 70
    ref = Ref(P, H, page, d, seed=d)
    cache = ref.to(DEV)
    slots = torch.randperm(P * page, generator=torch.Generator().manual_seed(page))[:T].tolist()
    slots = (slots + [-1] * T)[:T]
    slots[3], slots[T - 1] = -1, -5
    kv = torch.stack((normal((T, H, d), dtype, 1, 3.0), close((T, H, d), dtype, 2)), 1)
    kv[5, 0] = bits((H, d), dtype, 3)
    kv[6] = 0.0
    kv[7] = -0.0
    kv[8, :, :, ::2] = -0.0
    gpu = kv.to(DEV)
    fa.fa_cache4_write(cache, gpu[:, 0], gpu[:, 1], i32(slots))
    ref.write(kv[:, 0], kv[:, 1], slots)
    same(cache, ref)
    assert status() == 0


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("kind", [bits, close])
def test_write_every_rounding(dtype, kind):
    """A million values of each kind."""
    P, H, page, d = 40, 2, 128, 128
    ref = Ref(P, H, page, d)
    cache = ref.to(DEV)
    k, v = kind((P * page, H, d), dtype, 11), kind((P * page, H, d), dtype, 12)
    slots = list(range(P * page))
    fa.fa_cache4_write(cache, k.to(DEV), v.to(DEV), i32(slots))
    from cache4_util import encode
    for x, code, scale in ((k, ref.k, ref.k_scale), (v, ref.v, ref.v_scale)):
        c, s = encode(x)
        code.copy_(c.unflatten(0, (P, page)).transpose(1, 2))
        scale.copy_(s.unflatten(0, (P, page)).transpose(1, 2))
    same(cache, ref)


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
def test_write_every_largest_value(dtype):
    """Every 16-bit magnitude as the largest of a block, the rest on borders of its scale."""
    n = 0x7C00 if dtype == "fp16" else 0x7F80
    top = torch.arange(n, dtype=torch.int32).to(torch.int16).view(DTYPES[dtype])
    x = torch.zeros(n, 16, dtype=torch.float64)
    x[:, 0] = top.double()
    for i, part in enumerate((0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 0.26, 0.74, 1.26, 1.74, 2.51, 3.49, 4.99, 5.01), 1):
        x[:, i] = top.double() * part / 6 * (-1) ** i
    x = torch.where(x.abs() <= top.double()[:, None], x, 0.0).to(DTYPES[dtype])
    d, page = 128, 128
    x = torch.cat((x, x[:-n % 1024 or None][:(-n) % 1024])) if n % 1024 else x
    x = x.reshape(-1, 1, d)
    P = -(-x.shape[0] // page)
    ref = Ref(P, 1, page, d)
    cache = ref.to(DEV)
    slots = list(range(x.shape[0]))
    fa.fa_cache4_write(cache, x.to(DEV), x.to(DEV), i32(slots))
    ref.write(x, x, slots)
    same(cache, ref)


@pytest.mark.parametrize("T", [1, 2, 31, 33, 1000])
def test_write_sizes_and_strides(T):
    """Lengths around a block's tokens; head-major rows, one row for all tokens (stride 0)."""
    H, page, d = 4, 64, 96
    P = -(-T // page) + 1
    slots = [(7 * t) % (P * page) if P * page % 7 else t for t in range(T)]
    for make in (lambda x: x, lambda x: x.transpose(0, 1).contiguous().transpose(0, 1), lambda x: x[:1].expand(T, H, d)):
        ref = Ref(P, H, page, d, seed=T)
        cache = ref.to(DEV)
        k, v = make(normal((T, H, d), "bf16", 1)), make(normal((T, H, d), "bf16", 2))
        fa.fa_cache4_write(cache, make(normal((T, H, d), "bf16", 1).to(DEV)), make(normal((T, H, d), "bf16", 2).to(DEV)), i32(slots))
        ref.write(k, v, slots)
        same(cache, ref)


def test_write_slots_that_are_none():
    ref = Ref(3, 2, 16, 32)
    cache = ref.to(DEV)
    k, v = normal((6, 2, 32), "fp16", 1), normal((6, 2, 32), "fp16", 2)
    slots = [5, 48, -1, -2 ** 31, 2 ** 31 - 1, 47]
    fa.fa_cache4_write(cache, k.to(DEV), v.to(DEV), i32(slots))
    assert status() == 6
    ref.write(k, v, slots)
    same(cache, ref)
    fa.fa_cache4_write(cache, k[:4].to(DEV), v[:4].to(DEV), i32([-1] * 4))
    fa.fa_cache4_write(cache, k[:0].to(DEV), v[:0].to(DEV), i32([]))
    same(cache, ref)
    assert status() == 0
    # the same slot twice: some of one or the other, and nothing beside it
    fa.fa_cache4_write(cache, k[:2].to(DEV), v[:2].to(DEV), i32([9, 9]))
    got = cache.data.cpu()
    ref.write(k[:1], v[:1], [9])
    one = ref.bytes()
    ref.write(k[1:2], v[1:2], [9])
    assert ((got == one) | (got == ref.bytes())).all()


# ---------------------------------------------------------------------------
# reading back


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("d", [32, 64, 96, 128])
@pytest.mark.parametrize("page", [16, 32, 64, 128])
def test_read(dtype, d, page):
    lens, N = [0, 1, page, 2 * page + 5, 100, -3, 10 ** 6], 150
    table, pool = pages_for([0, 1, page, 2 * page + 5, 100, 0, 3 * page], page, d)
    ref = Ref(pool, 2, page, d, seed=page, lowest=0, highest=0xE3)
    cache = ref.to(DEV)
    k, v = fa.fa_cache4_read(cache, table.to(DEV), i32(lens), N, dtype=DTYPES[dtype])
    want = ref.read(table, lens, N, DTYPES[dtype])
    assert torch.equal(k.cpu(), want[0]) and torch.equal(v.cpu(), want[1])
    assert status() == 6  # two lengths that are none, and places without a page


def test_read_bad_pages_and_given_outputs():
    page, d = 16, 64
    table, pool = pages_for([40, 30], page, 1)
    ref = Ref(pool, 3, page, d)
    cache = ref.to(DEV)
    table[0, 1], table[1, 0] = pool, -1
    wide = torch.full((2, table.shape[1] + 5), 1, dtype=torch.int32)
    wide[:, :table.shape[1]] = table
    k, v = (torch.full((2, 3, 37, d), 7.0, dtype=torch.float16, device=DEV) for _ in range(2))
    got = fa.fa_cache4_read(cache, wide.to(DEV)[:, :table.shape[1]], i32([40, 30]), 37, k=k, v=v)
    want = ref.read(table, [40, 30], 37, torch.float16)
    assert got[0] is k and torch.equal(k.cpu(), want[0]) and torch.equal(v.cpu(), want[1])
    assert status() == 6


def test_read_into_outputs_on_odd_16_bytes():
    """Rows that begin 16 bytes behind a 32-byte border, one output or both."""
    page, d, N = 32, 96, 50
    table, pool = pages_for([50, 20], page, 1)
    ref = Ref(pool, 2, page, d)
    n = 2 * 2 * N * d
    want = ref.read(table, [50, 20], N, torch.bfloat16)
    for shift_k, shift_v in ((8, 0), (0, 8), (8, 8)):
        bufs = [torch.full((n + 16,), 7.0, dtype=torch.bfloat16, device=DEV) for _ in range(2)]
        k, v = (x[s:s + n].view(2, 2, N, d) for x, s in zip(bufs, (shift_k, shift_v)))
        fa.fa_cache4_read(ref.to(DEV), table.to(DEV), i32([50, 20]), N, k=k, v=v)
        assert torch.equal(k.cpu(), want[0]) and torch.equal(v.cpu(), want[1])
        for x, s in zip(bufs, (shift_k, shift_v)):
            assert (x[:s] == 7).all() and (x[s + n:] == 7).all()


# ---------------------------------------------------------------------------
# attention


def attend(ref, table, lens, q, causal=False, scale=None, **kw):
    o, lse = fa.fa_decode_cache4(q.to(DEV), ref.to(DEV), table.to(DEV), i32(lens), causal=causal, scale=scale, **kw)
    within(o, lse, attend_bounds(ref, q, table, lens, q.shape[-1] ** -0.5 if scale is None else scale, causal))
    return o, lse


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("d", [32, 64, 96, 128])
@pytest.mark.parametrize("page", [16, 32, 64, 128])
@pytest.mark.parametrize("G,Nq", [(1, 1), (4, 1), (8, 1), (1, 16), (3, 3), (16, 4), (7, 16)])
def test_attend(dtype, d, page, G, Nq):
    """Mixed lengths: none, one, ends inside tiles and pages, several stages."""
    H = 2
    lens = [0, 1, 17, 64, 130, 257, max(Nq, 3)]
    table, pool = pages_for(lens, page, G)
    ref = Ref(pool, H, page, d, seed=Nq)
    q = normal((len(lens), H * G, Nq, d), dtype, d + G)
    for causal in (False, True):
        attend(ref, table, lens, q, causal)
    assert status() == 0


@pytest.mark.parametrize("d,page,H,G,Nq,lens,causal", [
    (128, 64, 8, 4, 1, [5000, 1, 777], False), (128, 16, 2, 8, 1, [6001], False), (64, 16, 4, 1, 1, [3000, 4100], False),
    (128, 32, 1, 4, 4, [4099, 3, 64], True), (32, 128, 3, 2, 2, [4000, 129], True), (96, 64, 2, 4, 4, [3001, 2000], True),
    (96, 16, 1, 1, 1, [6000], False), (64, 128, 1, 16, 16, [1500, 20], True), (128, 128, 1, 32, 4, [1000, 5, 300], True),
    (128, 64, 32, 1, 1, [700] * 5 + [64] * 20, False), (32, 16, 32, 1, 1, [300 + 7 * i for i in range(24)], False),
], ids=str)
def test_attend_long(d, page, H, G, Nq, lens, causal):
    """Runs of work that begin and end inside sequences, and their merge."""
    table, pool = pages_for(lens, page, 3)
    ref = Ref(pool, H, page, d, seed=5)
    attend(ref, table, lens, normal((len(lens), H * G, Nq, d), "bf16", 6), causal)
    assert status() == 0


@pytest.mark.parametrize("d", [32, 64, 96, 128])
@pytest.mark.parametrize("page", [16, 64, 128])
def test_what_lies_behind_the_end(d, page):
    """Slots behind the last key hold any bytes, scales among them that are infinite or NaN as fp16: no row sees them."""
    lens, Nq = [1, 5, 16, 37, 130], 4
    table, pool = pages_for(lens, page, 2)
    ref = Ref(pool, 2, page, d, seed=1)
    q = normal((len(lens), 6, Nq, d), "fp16", 2)
    for causal in (False, True):
        want = attend_bounds(ref, q, table, lens, d ** -0.5, causal)
        ref2 = Ref(pool, 2, page, d, seed=1)
        for b, n in enumerate(lens):
            for at in range(n, table.shape[1] * page):
                p = int(table[b, at // page])
                if p >= 0:
                    for code, scale in ((ref2.k, ref2.k_scale), (ref2.v, ref2.v_scale)):
                        code[p, :, at % page] = 7
                        scale[p, :, at % page] = 0xF8 if at % 2 else 0xFF
        o, lse = fa.fa_decode_cache4(q.to(DEV), ref2.to(DEV), table.to(DEV), i32(lens), causal=causal)
        within(o, lse, want)
    # and in 16 bits, where they become zeros
    k, v = fa.fa_cache4_read(ref2.to(DEV), table.to(DEV), i32(lens), 140)
    want = ref2.read(table, lens, 140, torch.bfloat16)
    assert torch.equal(k.cpu(), want[0]) and torch.equal(v.cpu(), want[1])


def test_rows_that_see_nothing():
    """Fewer keys than causal queries, and sequences without any."""
    lens, Nq, d = [0, 1, 2, 5], 6, 64
    table, pool = pages_for(lens, 16, 4)
    ref = Ref(pool, 2, 16, d)
    o, lse = attend(ref, table, lens, normal((4, 4, Nq, d), "bf16", 1), True)
    assert torch.isneginf(lse[0]).all() and torch.isneginf(lse[1, :, :5]).all() and (o[1, :, :5] == 0).all()


def test_bad_pages_and_lengths():
    lens = [100, 60, 33, -4, 10 ** 6]
    table, pool = pages_for([100, 60, 33, 0, 112], 16, 4)
    ref = Ref(pool, 2, 16, 128)
    table[0, 2], table[1, 0], table[2, :] = pool, -1, 2 ** 31 - 1
    attend(ref, table, lens, normal((5, 8, 1, 128), "fp16", 1))
    assert status() == 6


@pytest.mark.parametrize("scale_bytes", [(0, 8), (0, 0xE3), (0xD8, 0xE3), (0x30, 0x38)])
def test_scales_of_any_size(scale_bytes):
    """Zero and subnormal scales, the largest, and all of them side by side."""
    lens, d = [300, 47], 128
    table, pool = pages_for(lens, 32, 4)
    ref = Ref(pool, 1, 32, d, lowest=scale_bytes[0], highest=scale_bytes[1])
    big = scale_bytes[1] == 0xE3
    if big:  # K as usual: scores beyond fp32's exponentials say nothing
        ref.k_scale = torch.randint(0x50, 0x70, ref.k_scale.shape)
    for dtype in ("fp16", "bf16"):
        q = normal((2, 4, 1, d), dtype, 2)
        if big and dtype == "fp16":
            q = q * 1.0
        attend(ref, table, lens, q)


@pytest.mark.parametrize("d", [64, 128])
def test_sink(d):
    """A key with 0.9999 of the weight and V = 0: the others' small weights are kept."""
    n, H, G = 4096, 2, 4
    table, pool = pages_for([n], 64, 4)
    ref = Ref(pool, H, 64, d, seed=2, lowest=0x40, highest=0x48)
    x = torch.sign(torch.randn(d, generator=torch.Generator().manual_seed(1)))
    q = x.expand(1, H * G, 1, d).to(torch.bfloat16).contiguous()
    p, slot = int(table[0, 3]), 17
    ref.v[p, :, slot] = 0
    k, _, _ = ref.rows(table[0], n)
    rest = torch.logsumexp((k @ x.double()) * d ** -0.5, -1).max()
    per = float(rest + math.log(1e4)) * d ** 0.5 / d        # of every channel, along q
    ref.k[p, :, slot] = (5 + 8 * (x < 0)).long()            # 3 or -3, by a scale that reaches it
    from cache4_util import SCALES
    ref.k_scale[p, :, slot] = int(torch.searchsorted(SCALES, torch.tensor(per / 3, dtype=torch.float64)))
    o, _ = attend(ref, table, [n], q)
    assert o.abs().max() > 0


@pytest.mark.parametrize("by", [0.0, 8.0, 300.0])
def test_scores_of_any_size(by):
    """Queries of zeros, scores of some hundred, and a reference that moves again and again."""
    lens, d = [700, 40], 64
    table, pool = pages_for(lens, 16, 4)
    ref = Ref(pool, 2, 16, d, seed=7, lowest=0x40, highest=0x78)
    q = normal((2, 8, 2, d), "bf16", 3, by)
    attend(ref, table, lens, q, True)
    order = torch.arange(700) / 700.0        # keys that grow along the sequence
    ref.k_scale[table[0, torch.arange(700) // 16].long(), :, torch.arange(700) % 16] = (0x40 + 0x38 * order).long()[:, None, None].expand(-1, 2, d // 16)
    attend(ref, table, lens, q, True)


@pytest.mark.parametrize("G,Nq", [(4, 1), (8, 1), (4, 4)])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_queries_that_are_not_finite(G, Nq, bad):
    """A row with such a channel is NaN (or nothing); the other rows of its KV head, causal ones among them, are as ever."""
    lens, d = [300, 41], 64
    table, pool = pages_for(lens, 32, 4)
    ref = Ref(pool, 2, 32, d)
    q = normal((2, 2 * G, Nq, d), "bf16", 3)
    want = attend_bounds(ref, q, table, lens, d ** -0.5, True)
    x = q.clone()
    x[:, 1, Nq - 1, 5], x[:, G + 2, 0, 9] = bad, bad
    o, lse = fa.fa_decode_cache4(x.to(DEV), ref.to(DEV), table.to(DEV), i32(lens), causal=True)
    hit = torch.zeros(2, 2 * G, Nq, dtype=torch.bool)
    hit[:, 1, Nq - 1], hit[:, G + 2, 0] = True, True
    assert not torch.isfinite(lse.cpu()[hit]).any()
    o, lse = o.cpu().double(), lse.cpu().double()
    assert ((o - want[0]).abs() <= want[2])[~hit].all() and ((lse - want[1]).abs() <= want[3])[~hit].all()


@pytest.mark.parametrize("R", [1, 2, 3, 4, 5, 8, 9, 16, 17, 32, 33, 64, 65, 100])
def test_every_layout_of_rows(R):
    """One KV head with R query heads: four, eight and sixteen rows a warp, warps along the rows, groups of 64."""
    lens, d = [1500, 0, 77, 400], 128
    table, pool = pages_for(lens, 64, R)
    ref = Ref(pool, 1, 64, d, seed=R)
    attend(ref, table, lens, normal((4, R, 1, d), "fp16", R))
    attend(ref, table[2:], lens[2:], normal((2, R, 1, d), "fp16", R))


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("d", [96, 128])
@pytest.mark.parametrize("page", [16, 32, 64, 128])
@pytest.mark.parametrize("G,Nq", [(33, 1), (12, 3), (16, 4), (9, 16), (4, 10), (17, 1), (6, 4), (8, 4)])
def test_many_rows(dtype, d, page, G, Nq):
    """Groups of 32 or 64 rows, whole segments and shared ones, the last group not full."""
    for lens in ([3000, 0, 1, 129, 700], [300, 128, 5], [40] * 90):
        table, pool = pages_for(lens, page, 5)
        ref = Ref(pool, 2, page, d, seed=6)
        attend(ref, table, lens, normal((len(lens), 2 * G, Nq, d), dtype, 7), Nq > 1)
    assert status() == 0


@pytest.mark.parametrize("d", [96, 128])
@pytest.mark.parametrize("G", [20, 11])
@pytest.mark.parametrize("by", [0.0, 8.0, 300.0])
def test_many_rows_scores_of_any_size(d, G, by):
    lens = [1500, 140]
    table, pool = pages_for(lens, 16, 4)
    ref = Ref(pool, 2, 16, d, seed=7, lowest=0x40, highest=0x78)
    q = normal((2, 2 * G, 2, d), "bf16", 3, by)
    attend(ref, table, lens, q, True)
    at = torch.arange(1500)                  # keys that grow along the sequence
    ref.k_scale[table[0, at // 16].long(), :, at % 16] = (0x40 + 0x38 * (at / 1500.0)).long()[:, None, None].expand(-1, 2, d // 16)
    attend(ref, table, lens, q, True)


@pytest.mark.parametrize("d", [96, 128])
@pytest.mark.parametrize("G", [20, 14])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_many_rows_queries_that_are_not_finite(d, G, bad):
    lens, Nq = [300, 41], 2
    table, pool = pages_for(lens, 32, 4)
    ref = Ref(pool, 2, 32, d)
    q = normal((2, 2 * G, Nq, d), "bf16", 3)
    want = attend_bounds(ref, q, table, lens, d ** -0.5, True)
    x = q.clone()
    x[:, 1, Nq - 1, 5], x[:, G + 12, 0, 9] = bad, bad
    o, lse = fa.fa_decode_cache4(x.to(DEV), ref.to(DEV), table.to(DEV), i32(lens), causal=True)
    hit = torch.zeros(2, 2 * G, Nq, dtype=torch.bool)
    hit[:, 1, Nq - 1], hit[:, G + 12, 0] = True, True
    assert not torch.isfinite(lse.cpu()[hit]).any()
    o, lse = o.cpu().double(), lse.cpu().double()
    assert ((o - want[0]).abs() <= want[2])[~hit].all() and ((lse - want[1]).abs() <= want[3])[~hit].all()


@pytest.mark.parametrize("d", [96, 128])
@pytest.mark.parametrize("page", [16, 64, 128])
@pytest.mark.parametrize("G", [10, 5])
def test_many_rows_what_lies_behind_the_end(d, page, G):
    """... and pages that are none, and lengths that are cut."""
    lens, Nq = [1, 37, 130, 1000, 10 ** 6], 4
    short = [min(n, 1100) for n in lens]
    table, pool = pages_for(short, page, 2)
    ref = Ref(pool, 2, page, d, seed=1)
    for b, n in enumerate(short):
        if n % page:
            last = table[b, n // page].long()
            for x in (ref.k_scale, ref.v_scale):
                x[last, :, n % page:] = 0xFF
    if short[-1] % page:                        # cut to the table's places, the last of which hold none
        ref.k_scale[table[-1, short[-1] // page].long()] = 0x60
        ref.v_scale[table[-1, short[-1] // page].long()] = 0x60
    table[3, 2], table[3, 0] = -1, 2 ** 31 - 1
    attend(ref, table, lens, normal((5, 2 * G, Nq, d), "fp16", 2), True)
    assert status() == 6


def test_many_rows_twice_the_same_and_on_two_streams():
    lens = [3000, 17, 900, 64]
    table, pool = pages_for(lens, 32, 4)
    ref = Ref(pool, 4, 32, 128)
    cache, t, n = ref.to(DEV), table.to(DEV), i32(lens)
    q = normal((4, 64, 4, 128), "bf16", 1).to(DEV)
    want = fa.fa_decode_cache4(q, cache, t, n, causal=True)
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    outs = [[fa.fa_decode_cache4(q, cache, t, n, causal=True, stream=s) for _ in range(5)] for s in streams]
    torch.cuda.synchronize()
    for o, lse in outs[0] + outs[1]:
        assert torch.equal(o, want[0]) and torch.equal(lse, want[1])


def test_more_segments_than_blocks():
    """Short sequences, more of them with their heads than blocks: runs over many whole segments."""
    lens = [(37 * b) % 140 for b in range(200)]
    table, pool = pages_for(lens, 16, 2)
    ref = Ref(pool, 4, 16, 32, seed=1)
    attend(ref, table, lens, normal((200, 8, 1, 32), "bf16", 2))
    lens = [1] * 700 + [0] * 20 + [300] * 3
    table, pool = pages_for(lens, 128, 2)
    ref = Ref(pool, 1, 128, 64, seed=1)
    attend(ref, table, lens, normal((723, 1, 2, 64), "fp16", 2), True)
    assert status() == 0


@pytest.mark.parametrize("d", [32, 64, 96, 128])
@pytest.mark.parametrize("page", [16, 32, 64, 128])
@pytest.mark.parametrize("G,Nq", [(1, 1), (4, 1), (1, 3), (8, 1), (2, 4), (5, 1)])
def test_a_warp_a_segment(d, page, G, Nq):
    """More segments than any grid of blocks, of up to 256 keys: what lies behind the last key is no number."""
    lens = [0, 1, 2, 3, 15, 16, 17, 31, 32, 33, 63, 64, 65, 255, 256] + [(53 * b) % 257 for b in range(155)]
    table, pool = pages_for(lens, page, 5)
    ref = Ref(pool, 4, page, d, seed=6)
    for b, n in enumerate(lens):
        if n % page:
            last = table[b, n // page].long()
            ref.k_scale[last, :, n % page:] = 0xFF
            ref.v_scale[last, :, n % page:] = 0xFF
    attend(ref, table, lens, normal((170, 4 * G, Nq, d), "bf16" if G > 2 else "fp16", 7), Nq > 1)
    assert status() == 0


def test_a_warp_a_segment_of_many_pages():
    lens = [1 + 11 * b % 600 for b in range(400)]
    table, pool = pages_for(lens, 16, 3)
    ref = Ref(pool, 4, 16, 64, seed=4)
    attend(ref, table, lens, normal((400, 8, 1, 64), "fp16", 5))
    assert status() == 0


def test_a_warp_a_segment_bad_pages_and_lengths():
    lens = [100, 60, 33, -4, 10 ** 6] + [20] * 700
    table, pool = pages_for([min(n, 112) for n in lens], 16, 4)
    ref = Ref(pool, 1, 16, 128)
    table[0, 2], table[1, 0], table[2, :], table[3:5, 3], table[9, 1] = pool, -1, 2 ** 31 - 1, -2 ** 31, -1
    attend(ref, table, lens, normal((705, 8, 1, 128), "fp16", 1))
    assert status() == 6


def test_query_strides_scale_and_given_outputs():
    d, lens = 128, [90, 200]
    table, pool = pages_for(lens, 64, 4)
    ref = Ref(pool, 2, 64, d)
    wide = normal((2, 3, 20, d), "fp16", 5)
    q = wide[:, :, 4:12].transpose(1, 2)              # [B, heads, Nq, d] inside [B, Nq, heads, d]
    gpu = wide.to(DEV)[:, :, 4:12].transpose(1, 2)
    o = torch.full((2, 8, 3, d), 9.0, dtype=torch.float16, device=DEV)
    lse = torch.full((2, 8, 3), 9.0, device=DEV)
    ws = torch.empty(fa.fa_decode_cache4_workspace_size(2, 8, 2, 3, d), dtype=torch.uint8, device=DEV)
    got = fa.fa_decode_cache4(gpu, ref.to(DEV), table.to(DEV), i32(lens), o=o, lse=lse, scale=0.2, causal=True, workspace=ws)
    assert got[0] is o and got[1] is lse
    within(o, lse, attend_bounds(ref, q, table, lens, 0.2, True))
    alone, none = fa.fa_decode_cache4(gpu, ref.to(DEV), table.to(DEV), i32(lens), scale=0.2, causal=True, return_lse=False)
    assert none is None and torch.equal(alone, o)
    zero, lse0 = fa.fa_decode_cache4(gpu, ref.to(DEV), table.to(DEV), i32(lens), scale=0.0)
    within(zero, lse0, attend_bounds(ref, q, table, lens, 0.0, False))


@pytest.mark.parametrize("lens,Nq", [([3000, 17, 900], 1), ([64, 1], 4), ([500] * 40, 2)])
def test_twice_the_same_and_on_two_streams(lens, Nq):
    """No order of summation is left to chance; two calls at once with a workspace each."""
    table, pool = pages_for(lens, 32, 4)
    ref = Ref(pool, 4, 32, 128)
    cache, t, n = ref.to(DEV), table.to(DEV), i32(lens)
    q = normal((len(lens), 16, Nq, 128), "bf16", 1).to(DEV)
    want = fa.fa_decode_cache4(q, cache, t, n, causal=True)
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    outs = [[fa.fa_decode_cache4(q, cache, t, n, causal=True, stream=s) for _ in range(5)] for s in streams]
    torch.cuda.synchronize()
    for o, lse in outs[0] + outs[1]:
        assert torch.equal(o, want[0]) and torch.equal(lse, want[1])


def test_graph_follows_lengths_and_tables():
    """A captured step replays with the lengths, pages and codes of the moment; two graphs share a workspace."""
    page, d, H = 16, 64, 2
    table, pool = pages_for([400, 60], page, 4)
    ref = Ref(pool, H, page, d)
    cache, t, n = ref.to(DEV), table.to(DEV), i32([0, 0])
    q = normal((2, 8, 1, d), "fp16", 1)
    gpu = q.to(DEV)
    ws = torch.empty(fa.fa_decode_cache4_workspace_size(2, 8, H, 1, d), dtype=torch.uint8, device=DEV)
    graphs, outs = [], []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(fa.fa_decode_cache4(gpu, cache, t, n, workspace=ws))
        graphs.append(g)
    for lens in ([400, 60], [0, 1], [333, 0], [17, 59]):
        n.copy_(i32(lens))
        for g in graphs:
            g.replay()
        torch.cuda.synchronize()
        want = attend_bounds(ref, q, table, lens, d ** -0.5, False)
        for o, lse in outs:
            within(o, lse, want)
    assert status() == 0


def test_one_key():
    """One key: o is its value, whatever the query."""
    ref = Ref(2, 1, 16, 128, seed=3)
    table = torch.tensor([[1]], dtype=torch.int32)
    o, lse = attend(ref, table, [1], normal((1, 5, 1, 128), "bf16", 1))
    _, v, _ = ref.rows(table[0], 1)
    assert torch.equal(o.cpu().double(), v[0, 0].expand(1, 5, 1, 128))


def test_offsets_beyond_32_bits():
    """A cache of more than 2^32 bytes: pages at its end are written, read and attended to."""
    H, page, d = 8, 128, 128
    P = (2 ** 32 // (H * page * 144)) + 700
    data = torch.zeros((P, H, page, 144), dtype=torch.uint8, device=DEV)
    cache = fa.FACache4(data)
    lens = [200, 130]
    table = torch.tensor([[P - 1, 3], [P - 2, P - 3]], dtype=torch.int32)
    T = sum(lens)
    pos = [(b, t) for b, n in enumerate(lens) for t in range(n)]
    slots = [int(table[b, t // page]) * page + t % page for b, t in pos]
    k, v = normal((T, H, d), "bf16", 1), normal((T, H, d), "bf16", 2)
    fa.fa_cache4_write(cache, k.to(DEV), v.to(DEV), i32(slots))
    small = Ref(4, H, page, d)
    near = torch.tensor([[0, 1], [2, 3]], dtype=torch.int32)
    small.write(k, v, [int(near[b, t // page]) * page + t % page for b, t in pos])
    q = normal((2, H, 1, d), "bf16", 3)
    o, lse = fa.fa_decode_cache4(q.to(DEV), cache, table.to(DEV), i32(lens))
    within(o, lse, attend_bounds(small, q, near, lens, d ** -0.5, False))
    rk, rv = fa.fa_cache4_read(cache, table.to(DEV), i32(lens), 200)
    want = small.read(near, lens, 200, torch.bfloat16)
    assert torch.equal(rk.cpu(), want[0]) and torch.equal(rv.cpu(), want[1])
    assert int(torch.count_nonzero(data[4:P - 3])) == 0
