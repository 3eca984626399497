"""The 8-bit paged cache on the GPU (fa_cache_write, fa_cache_read,
fa_cache_select, fa_decode_cache) against its definition in 64 bits
(cache_util).  Writing, reading and selecting are compared for equality,
attention within the bounds derived there."""
import math

import pytest
import torch

from cache_util import CODES, DTYPES, Ref, bounds, pages_for

pytestmark = pytest.mark.gpu

FA_ERR_BOUNDS = 6


@pytest.fixture(scope="module")
def fa():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import attention_forward_02_gb300 as fa
    status(fa)
    return fa


def status(fa):
    return fa.fa_last_device_status(torch.cuda.current_stream().cuda_stream)


def dev(x):
    return torch.as_tensor(x, dtype=torch.int32).cuda()


def randn(shape, dtype, seed, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * scale).to(dtype)


def same_values(got, want):
    """Equality of code values or scales, NaN equal to NaN."""
    return torch.equal(torch.nan_to_num(got.cpu().double(), nan=1e9), torch.nan_to_num(want.double(), nan=1e9))


def check_cache(cache, ref, means=True):
    names = ["k", "v", "k_scale", "v_scale"] + (["k_mean", "k_mean_scale"] if means else [])
    for name in names:
        got = getattr(cache, name)
        got = got.float() if name in ("k", "v") else got
        assert same_values(got, getattr(ref, name)), name


# ---------------------------------------------------------------------------
# writing


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("page,d,heads", [(16, 32, 3), (16, 96, 1), (32, 64, 2), (64, 128, 2), (64, 96, 1),
                                          (128, 128, 1), (128, 32, 2)])
def test_write(fa, fmt, dtype, page, d, heads):
    """Fresh pages, pages begun before, one token, none, exactly a page, several pages; then one more token each."""
    before = [0, 5, page - 1, 3, page, 2 * page + 7, 0, page // 2]
    new = [page, 1, 1, 0, 1, 3 * page, 2, page // 2]
    ends = [a + n + 1 for a, n in zip(before, new)]
    table, pool = pages_for(ends, page, 1)
    ref = Ref(pool, heads, page, d, fmt, 2)
    cache = ref.to("cuda")
    cu = [0]
    for n in new:
        cu.append(cu[-1] + n)
    # rows behind the last sequence's are ignored
    k, v = (randn((cu[-1] + 5, heads, d), DTYPES[dtype], s, 3.0) for s in (3, 4))
    fa.fa_cache_write(cache, k.cuda(), v.cuda(), dev(table), dev(before), cu_seqlens=dev(cu))
    assert status(fa) == 0
    ref.write(k, v, table, before, cu)
    check_cache(cache, ref)
    lens = [a + n for a, n in zip(before, new)]
    k, v = (randn((len(lens), heads, d), DTYPES[dtype], s, 40.0) for s in (5, 6))  # scales grow: codes move
    fa.fa_cache_write(cache, k.cuda(), v.cuda(), dev(table), dev(lens))
    assert status(fa) == 0
    ref.write(k, v, table, lens, list(range(len(lens) + 1)))
    check_cache(cache, ref)


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
def test_write_special_values(fa, fmt):
    """Infinities saturate, NaN stays NaN (int8: 0), neither sets the scale; zeros; the smallest and largest numbers;
    amax just at and above the code's top."""
    page, d, heads = 16, 32, 1
    rows = torch.zeros(7 * page, heads, d)
    rows[page:2 * page] = randn((page, heads, d), torch.float32, 1)
    rows[page, 0, 3], rows[page + 1, 0, 4], rows[page + 2, 0, 5] = math.inf, -math.inf, math.nan
    rows[2 * page:3 * page] = math.nan
    rows[3 * page:4 * page] = randn((page, heads, d), torch.float32, 2, 2.0 ** -80)
    rows[4 * page:5 * page] = randn((page, heads, d), torch.float32, 3, 2.0 ** 125).clamp(-3e38, 3e38)
    rows[5 * page:6 * page] = torch.linspace(-1, 1, page * d).reshape(page, 1, d) * (448.0 if fmt == "e4m3" else 127.0)
    rows[6 * page:] = torch.linspace(-1, 1, page * d).reshape(page, 1, d) * (450.0 if fmt == "e4m3" else 127.5)
    k, v = rows.to(torch.bfloat16), rows.flip(0).to(torch.bfloat16)
    table, pool = pages_for([7 * page], page, 1)
    ref = Ref(pool, heads, page, d, fmt, 2)
    cache = ref.to("cuda")
    fa.fa_cache_write(cache, k.cuda(), v.cuda(), dev(table), dev([0]))
    assert status(fa) == 0
    ref.write(k, v, table, [0], [0, 7 * page])
    check_cache(cache, ref)


def test_write_strides_and_no_means(fa):
    """Rows out of one fused projection, and head-major rows; a cache without mean keys."""
    page, d, heads, T = 32, 64, 3, 70
    table, pool = pages_for([T], page, 1)
    for layout in ("fused", "heads"):
        ref = Ref(pool, heads, page, d, "e4m3", 2)
        cache = ref.to("cuda", means=False)
        if layout == "fused":
            qkv = randn((T, 5 * heads, d), torch.bfloat16, 3).cuda()
            k, v = qkv[:, 3 * heads:4 * heads], qkv[:, 4 * heads:]
        else:
            k = randn((heads, T, d), torch.bfloat16, 3).cuda().transpose(0, 1)
            v = randn((T, heads, 2 * d), torch.bfloat16, 4).cuda()[..., d:]
        fa.fa_cache_write(cache, k, v, dev(table), dev([0]))
        assert status(fa) == 0
        ref.write(k.cpu(), v.cpu(), table, [0], [0, T])
        check_cache(cache, ref, means=False)


def test_write_uneven_batch(fa):
    """One long sequence among single tokens: a grid for the mean length still writes all of its pages."""
    page, d, heads = 16, 32, 2
    new = [1] * 9 + [700] + [1] * 9
    before = [i % 20 for i in range(19)]
    table, pool = pages_for([a + n for a, n in zip(before, new)], page, 5)
    cu = [0]
    for n in new:
        cu.append(cu[-1] + n)
    ref = Ref(pool, heads, page, d, "int8", 6)
    cache = ref.to("cuda")
    k, v = (randn((cu[-1], heads, d), torch.float16, s) for s in (7, 8))
    fa.fa_cache_write(cache, k.cuda(), v.cuda(), dev(table), dev(before), cu_seqlens=dev(cu))
    assert status(fa) == 0
    ref.write(k, v, table, before, cu)
    check_cache(cache, ref)


@pytest.mark.parametrize("B", [32, 33, 128, 129, 300])
def test_write_many_sequences(fa, B):
    """Short sequences, runs of empty ones and a long one, in batches about the numbers that are counted at a time."""
    page, d, heads = 16, 32, 1
    new = [0 if i % 50 > 40 else (3 * i) % 7 for i in range(B)]
    new[B - 2], new[B - 1] = 90, 2
    before = [(5 * i) % 40 for i in range(B)]
    table, pool = pages_for([a + n for a, n in zip(before, new)], page, 5)
    cu = [0]
    for n in new:
        cu.append(cu[-1] + n)
    assert cu[-1] > B
    ref = Ref(pool, heads, page, d, "int8", 6)
    cache = ref.to("cuda")
    k, v = (randn((cu[-1], heads, d), torch.float16, s) for s in (7, 8))
    fa.fa_cache_write(cache, k.cuda(), v.cuda(), dev(table), dev(before), cu_seqlens=dev(cu))
    assert status(fa) == 0
    ref.write(k, v, table, before, cu)
    check_cache(cache, ref)


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("page,d,heads", [(16, 96, 2), (32, 32, 1), (128, 128, 1)])
def test_write_few_rows(fa, fmt, dtype, page, d, heads):
    """No more rows than sequences: single tokens, none, and the rows of others on one sequence; steps that complete
    pages, move codes to larger scales, and bring infinities and NaN."""
    new = [0] * 10 + [30] + [1] * 10 + [0] * 19
    before = [(7 * i) % (2 * page) for i in range(40)]
    before[10], before[11], before[12], before[13] = page - 7, page - 1, 2 * page - 1, page
    table, pool = pages_for([a + n + 8 for a, n in zip(before, new)], page, 5)
    cu = [0]
    for n in new:
        cu.append(cu[-1] + n)
    ref = Ref(pool, heads, page, d, fmt, 6)
    cache = ref.to("cuda")
    k, v = (randn((cu[-1], heads, d), DTYPES[dtype], s, 4.0) for s in (7, 8))
    k[3, 0, 1], k[33, 0, 2], v[31, 0, 3], v[34, 0, 0] = math.inf, math.nan, -math.inf, math.nan
    k[36] = math.nan
    fa.fa_cache_write(cache, k.cuda(), v.cuda(), dev(table), dev(before), cu_seqlens=dev(cu))
    assert status(fa) == 0
    ref.write(k, v, table, before, cu)
    check_cache(cache, ref)
    lens = [a + n for a, n in zip(before, new)]
    for step in range(6):  # a token each: pages end, scales grow
        k, v = (randn((40, heads, d), DTYPES[dtype], 20 + 2 * step + s, 2.0 ** (step - 2)) for s in (0, 1))
        fa.fa_cache_write(cache, k.cuda(), v.cuda(), dev(table), dev(lens))
        ref.write(k, v, table, lens, list(range(41)))
        lens = [n + 1 for n in lens]
    assert status(fa) == 0
    check_cache(cache, ref)


def test_write_few_rows_bad_pages(fa):
    """The same refusals on that way: bad page numbers, places behind the table, offsets that are none."""
    page, d = 16, 32
    table = torch.tensor([[0, 99], [-1, 1], [2, 3], [4, 5], [6, 7]], dtype=torch.int32)
    before = [16, 3, 40, 5, 31]
    ref = Ref(8, 1, page, d, "e4m3", 6)
    cache = ref.to("cuda")
    k, v = (randn((5, 1, d), torch.bfloat16, s) for s in (7, 8))
    fa.fa_cache_write(cache, k.cuda(), v.cuda(), dev(table), dev(before))
    assert status(fa) == FA_ERR_BOUNDS
    ref.write(k, v, table, before, list(range(6)))
    check_cache(cache, ref)
    fa.fa_cache_write(cache, k.cuda(), v.cuda(), dev(table), dev(before), cu_seqlens=dev([5, 4, 9, -3, 77, 6]))
    assert status(fa) == FA_ERR_BOUNDS
    check_cache(cache, ref)


def test_write_bad_pages(fa):
    """Tokens whose page number is bad, or whose place lies behind the table, are skipped and reported."""
    page, d, heads = 16, 32, 1
    table = torch.tensor([[0, 99, 1], [2, -1, 3], [4, 5, 6]], dtype=torch.int32)
    before, new = [0, 0, 40], [48, 48, 20]
    cu = [0, 48, 96, 116]
    ref = Ref(8, heads, page, d, "e4m3", 6)
    cache = ref.to("cuda")
    k, v = (randn((116, heads, d), torch.bfloat16, s) for s in (7, 8))
    fa.fa_cache_write(cache, k.cuda(), v.cuda(), dev(table), dev(before), cu_seqlens=dev(cu))
    assert status(fa) == FA_ERR_BOUNDS
    ref.write(k, v, table, before, cu)
    check_cache(cache, ref)
    # offsets that are none: nothing of those sequences is written
    cache = ref.to("cuda")
    fa.fa_cache_write(cache, k.cuda(), v.cuda(), dev([[0], [1], [2]]), dev([0, 0, 0]), cu_seqlens=dev([5, 2, 900, 90]))
    assert status(fa) == FA_ERR_BOUNDS
    check_cache(cache, ref)


# ---------------------------------------------------------------------------
# reading back


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("page,d", [(16, 32), (32, 96), (64, 64), (128, 128)])
@pytest.mark.parametrize("N", [1, 130, 500])
def test_read(fa, fmt, dtype, page, d, N):
    lens = [0, 1, page, 131, 470]
    table, pool = pages_for(lens, page, 1)
    ref = Ref(pool, 2, page, d, fmt, 2)
    if fmt == "e4m3":
        ref.k[int(table[3, 0]), 0, 0, 0] = math.nan
    k, v = fa.fa_cache_read(ref.to("cuda"), dev(table), dev(lens), N, dtype=DTYPES[dtype])
    assert status(fa) == 0
    for b, n in enumerate(lens):
        n = min(n, N)
        want = ref.sequence(table[b], n)
        for got, x in zip((k, v), want):
            assert same_values(got[b, :, :n], x.to(DTYPES[dtype]))
            assert not got[b, :, n:].any()


def test_read_bad_pages(fa):
    page, d = 16, 32
    table = torch.tensor([[0, 44, 1]], dtype=torch.int32)
    ref = Ref(3, 1, page, d, "e4m3", 2)
    k, v = fa.fa_cache_read(ref.to("cuda"), dev(table), dev([48]), 48)
    assert status(fa) == FA_ERR_BOUNDS
    for got, codes, scale in ((k, ref.k, ref.k_scale), (v, ref.v, ref.v_scale)):
        assert not got[0, 0, 16:32].any()
        assert same_values(got[0, 0, 32:], (codes[1, 0] * scale[1, 0]).to(torch.bfloat16))


# ---------------------------------------------------------------------------
# attention


def check_attention(fa, ref, q, table, lens, causal, pages=None, want_status=0, scale=None, got=None, **kw):
    d = q.shape[-1]
    scale = d ** -0.5 if scale is None else scale
    if got is None:
        got = fa.fa_decode_cache(q.cuda(), ref.to("cuda"), dev(table), dev(lens), causal=causal, scale=scale,
                                 pages=None if pages is None else dev(pages), **kw)
        assert status(fa) == want_status
    o, lse = (x.double().cpu() for x in got)
    eo, el, a, mag = ref.attend(q, table, lens, scale, causal, pages)
    n = max(1, max(lens))
    bo, bl = bounds(ref, q.dtype, eo, el, a, mag, n, d)
    empty = torch.isinf(el)
    assert torch.equal(empty, torch.isinf(lse) & (lse < 0))
    assert not o[empty].any()
    assert torch.isfinite(o).all()
    err, el_err = (o - eo).abs(), (lse - el).abs()[~empty]
    over, lse_over = float((err - bo).max()), float((el_err - bl[~empty]).max()) if el_err.numel() else 0.0
    assert over <= 0, "o off by up to %.3g, over its bound by %.3g" % (float(err.max()), over)
    assert lse_over <= 0, "lse off by up to %.3g, over its bound by %.3g" % (float(el_err.max()), lse_over)


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("d,page", [(32, 16), (64, 64), (96, 32), (128, 128), (128, 16)])
@pytest.mark.parametrize("heads,G,Nq", [(2, 1, 1), (1, 4, 1), (2, 8, 1), (1, 7, 3), (1, 16, 2), (1, 3, 16)])
def test_attention(fa, fmt, dtype, d, page, heads, G, Nq):
    lens = [1, 0, 15, 16, 17, 64, 129, 1000]
    table, pool = pages_for(lens, page, 1)
    ref = Ref(pool, heads, page, d, fmt, 2)
    q = randn((len(lens), heads * G, Nq, d), DTYPES[dtype], 3)
    for causal in (False, True):
        check_attention(fa, ref, q, table, lens, causal)


@pytest.mark.parametrize("G,Nq", [(40, 1), (16, 16), (70, 2)])
def test_attention_many_rows(fa, G, Nq):
    """More query rows a KV head than one block holds."""
    lens = [300, 20, 5]
    table, pool = pages_for(lens, 32, 1)
    ref = Ref(pool, 2, 32, 64, "e4m3", 2)
    q = randn((3, 2 * G, Nq, 64), torch.bfloat16, 3)
    check_attention(fa, ref, q, table, lens, True)


@pytest.mark.parametrize("d", [32, 64, 96, 128])
def test_attention_long(fa, d):
    """Long sequences beside short ones: parts of one sequence in many blocks, many sequences in one."""
    lens = [6000, 3, 1, 2500, 0, 777, 64, 65]
    table, pool = pages_for(lens, 64, 1)
    ref = Ref(pool, 1, 64, d, "e4m3", 2)
    q = randn((len(lens), 4, 1, d), torch.float16, 3)
    check_attention(fa, ref, q, table, lens, False)


def test_attention_many_sequences(fa):
    lens = [(37 * b) % 90 for b in range(700)]
    table, pool = pages_for(lens, 16, 1)
    ref = Ref(pool, 2, 16, 32, "int8", 2)
    q = randn((len(lens), 2, 1, 32), torch.float16, 3)
    check_attention(fa, ref, q, table, lens, False)


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
def test_attention_uneven_scales(fa, fmt):
    """Pages whose scales differ by many orders, rising and falling along the sequence."""
    lens = [640, 640]
    page = 16
    table, pool = pages_for(lens, page, 1)
    ref = Ref(pool, 2, page, 64, fmt, 2)
    for b, sign in ((0, 1), (1, -1)):
        for at in range(40):
            p = int(table[b, at])
            ref.v_scale[p] = 2.0 ** (sign * (at - 20))
            ref.k_scale[p] = 2.0 ** (-10 + at // 6)
    q = randn((2, 8, 1, 64), torch.bfloat16, 3)
    check_attention(fa, ref, q, table, lens, False)


@pytest.mark.parametrize("page", [16, 64])
def test_attention_scales_that_are_no_powers_of_two(fa, page):
    """A cache that something else has filled, with scales of any size (calibrated ones, say)."""
    lens = [333, 64]
    table, pool = pages_for(lens, page, 1)
    ref = Ref(pool, 2, page, 128, "int8", 2)
    g = torch.Generator().manual_seed(9)
    ref.k_scale, ref.v_scale = (torch.rand(ref.k_scale.shape, generator=g).float().double() * 0.03 + 0.01 for _ in range(2))
    for G in (4, 12):
        q = randn((2, 2 * G, 1, 128), torch.float16, 3)
        check_attention(fa, ref, q, table, lens, False)


def test_attention_peaked_and_rising(fa):
    """Scores with a wide spread, and scores that rise along the keys, so that the running reference moves."""
    lens = [900, 900]
    table, pool = pages_for(lens, 64, 1)
    ref = Ref(pool, 1, 64, 128, "int8", 2)
    q = randn((2, 8, 1, 128), torch.float16, 3)
    check_attention(fa, ref, q * 8, table, lens, False)
    for at in range(15):
        p = int(table[1, at])
        ref.k[p] = ref.k[p].abs()
        ref.k_scale[p] = 2.0 ** -9 * (1 if at < 5 else 2 if at < 10 else 4)
    check_attention(fa, ref, q.abs() * 4, table, lens, False)
    check_attention(fa, ref, q, table, lens, False, scale=0.0)


@pytest.mark.parametrize("scale", [2.0 ** -20, 2.0 ** 12])
def test_attention_query_magnitudes(fa, scale):
    """Query rows far from one, rows of zeros, and rows of one large and many small values."""
    lens = [200]
    table, pool = pages_for(lens, 32, 1)
    ref = Ref(pool, 1, 32, 64, "e4m3", 2)
    q = randn((1, 8, 1, 64), torch.bfloat16, 3) * scale
    q[0, 1] = 0
    q[0, 2, 0, 5] *= 1000
    check_attention(fa, ref, q, table, lens, False, scale=0.125 / scale)


@pytest.mark.parametrize("causal", [False, True])
def test_attention_garbage_behind_the_end(fa, causal):
    """Slots behind a sequence's end, and pages of nobody, hold NaN: none of it shows."""
    lens = [40, 1, 0, 100, 2]
    table, pool = pages_for(lens, 32, 1)
    ref = Ref(pool, 1, 32, 64, "e4m3", 2)
    used = torch.zeros(pool, 32, dtype=torch.bool)
    for b, n in enumerate(lens):
        for t in range(n):
            used[int(table[b, t // 32]), t % 32] = True
    for codes in (ref.k, ref.v):
        codes[:, 0][~used] = math.nan
    for scale in (ref.k_scale, ref.v_scale):
        scale[~used.any(1)] = math.nan
    q = randn((5, 4, 3, 64), torch.bfloat16, 3)
    check_attention(fa, ref, q, table, lens, causal)


def test_attention_nan_reaches_only_rows_that_see_it(fa):
    """A NaN value (or key) at the last position: the earlier causal queries do not see it, the last one does."""
    lens = [37]
    for name in ("k", "v"):
        table, pool = pages_for(lens, 16, 1)
        ref = Ref(pool, 1, 16, 64, "e4m3", 2)
        q = randn((1, 3, 4, 64), torch.bfloat16, 3)
        clean = ref.attend(q, table, lens, 0.125, True)[0]
        getattr(ref, name)[int(table[0, 2]), 0, 4, 7] = math.nan
        o, lse = fa.fa_decode_cache(q.cuda(), ref.to("cuda"), dev(table), dev(lens), causal=True, scale=0.125)
        o = o.double().cpu()
        assert torch.isfinite(o[:, :, :3]).all()
        assert (o[:, :, :3] - clean[:, :, :3]).abs().max() <= 2.0 ** -7 * clean.abs().max()
        assert torch.isnan(o[:, :, 3, 7]).all()
        if name == "k":
            assert torch.isnan(o[:, :, 3]).all() and torch.isnan(lse[:, :, 3]).all()


def test_attention_bad_pages_and_lengths(fa):
    """Bad page numbers are left out, a length behind the table is cut to it, a negative one is none."""
    page, d = 16, 64
    table = torch.tensor([[0, 99, 1], [-3, 2, 3], [4, 5, 6], [7, 7, 7]], dtype=torch.int32)
    ref = Ref(8, 2, page, d, "e4m3", 2)
    q = randn((4, 4, 1, d), torch.float16, 3)
    check_attention(fa, ref, q, table, [48, 40, 5000, -9], False, want_status=FA_ERR_BOUNDS)


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
@pytest.mark.parametrize("G,Nq,page", [(1, 1, 16), (8, 1, 64), (5, 3, 32), (20, 2, 16)])
def test_attention_listed_pages(fa, fmt, G, Nq, page):
    """Any list of pages: unordered, with negative entries, the partly filled last page or not, more slots than pages."""
    lens = [0, 5, 10 * page, 10 * page + 3, 4 * page - 1]
    table, pool = pages_for(lens, page, 1)
    ref = Ref(pool, 2, page, 64, fmt, 2)
    g = torch.Generator().manual_seed(5)
    pages = torch.full((len(lens), 2, Nq, 6), -1, dtype=torch.int32)
    for b, n in enumerate(lens):
        for h in range(2):
            for i in range(Nq):
                have = max(0, -(-(n - Nq + 1 + i) // page))
                row = torch.randperm(have, generator=g)[:6].int() if have else torch.zeros(0, dtype=torch.int32)
                pages[b, h, i, :len(row)] = row
                if len(row) > 3:
                    pages[b, h, i, 2] = -5
    q = randn((len(lens), 2 * G, Nq, 64), torch.bfloat16, 3)
    check_attention(fa, ref, q, table, lens, True, pages=pages)
    check_attention(fa, ref, q, table, lens, False, pages=pages)


@pytest.mark.parametrize("d", [32, 128])
def test_attention_many_listed_pages(fa, d):
    """Lists long enough that one query's pages go to many blocks, beside a sequence that has fewer pages than slots."""
    page, lens = 32, [6000, 500]
    table, pool = pages_for(lens, page, 1)
    ref = Ref(pool, 2, page, d, "e4m3", 2)
    g = torch.Generator().manual_seed(5)
    pages = torch.full((2, 2, 2, 120), -1, dtype=torch.int32)
    for h in range(2):
        for i in range(2):
            pages[0, h, i] = torch.randperm(6000 // page, generator=g)[:120].int()
            pages[1, h, i, :16] = torch.arange(16)
    q = randn((2, 12, 2, d), torch.float16, 3)
    check_attention(fa, ref, q, table, lens, False, pages=pages)


def test_calls_repeat_bit_for_bit_and_on_two_streams(fa):
    """The same call gives the same bits, alone and beside others on another stream with workspaces of their own."""
    lens = [3000, 17, 900]
    table, pool = pages_for(lens, 16, 1)
    ref = Ref(pool, 2, 16, 64, "e4m3", 2)
    cache, table, lens = ref.to("cuda"), dev(table), dev(lens)
    qs = [randn((3, 8, 2, 64), torch.bfloat16, s).cuda() for s in (3, 4)]

    def call(q):
        pages = fa.fa_cache_select(q, cache, table, lens, 20)
        return (pages, *fa.fa_decode_cache(q, cache, table, lens), *fa.fa_decode_cache(q, cache, table, lens, pages=pages))

    first = [call(q) for q in qs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in qs]
    got = [[], []]
    for _ in range(20):
        for k in range(2):
            with torch.cuda.stream(streams[k]):
                got[k].append(call(qs[k]))
    torch.cuda.synchronize()
    for k in range(2):
        for again in got[k]:
            assert all(torch.equal(x, y) for x, y in zip(again, first[k]))
    assert status(fa) == 0


def test_both_ways_through_python(fa, monkeypatch):
    """The CPython module's way and the longer one give the same results, in new memory and in given one, and refuse
    the same calls."""
    from attention_forward_02_gb300 import cache as module
    from attention_forward_02_gb300._lib import load
    assert module._quick(), "the CPython module is not built"
    lens = [300, 1, 0, 77]
    table, pool = pages_for([n + 1 for n in lens], 16, 1)
    ref = Ref(pool, 2, 16, 64, "e4m3", 2)
    table, new = dev(table), randn((4, 2, 64), torch.float16, 3).cuda()
    q = randn((4, 6, 2, 64), torch.float16, 4).cuda()

    def everything():
        cache, n = ref.to("cuda"), dev(lens)
        fa.fa_cache_write(cache, new, new, table, n)
        fa.fa_cache_write(cache, new, new, table, n, cu_seqlens=dev([0, 0, 1, 3, 4]))
        n += 1
        pages = fa.fa_cache_select(q, cache, table, n, 5, 2, 1, True)
        given = (torch.empty_like(q), torch.empty(4, 6, 2, device="cuda"), torch.empty_like(pages),
                 *(torch.empty(4, 2, 90, 64, dtype=torch.float16, device="cuda") for _ in range(2)))
        ws = torch.empty(1 << 26, dtype=torch.uint8, device="cuda")
        out = [*cache, pages, *fa.fa_decode_cache(q, cache, table, n), *fa.fa_cache_read(cache, table, n, 90)]
        a = fa.fa_decode_cache(q, cache, table, n, pages, given[0], given[1], 0.5, True, True, ws)
        b = fa.fa_cache_select(q, cache, table, n, 5, 2, 1, True, given[2], ws)
        c = fa.fa_cache_read(cache, table, n, 90, k=given[3], v=given[4])
        assert a[0] is given[0] and a[1] is given[1] and b is given[2] and c[0] is given[3] and c[1] is given[4]
        assert fa.fa_decode_cache(q, cache, table, n, return_lse=False)[1] is None
        bad = (lambda: fa.fa_decode_cache(q[:3], cache, table, n), lambda: fa.fa_decode_cache(q.float(), cache, table, n),
               lambda: fa.fa_decode_cache(q, cache, table.long(), n), lambda: fa.fa_decode_cache(q, cache, table, n.cpu()),
               lambda: fa.fa_decode_cache(q, cache._replace(v=cache.v[1:]), table, n),
               lambda: fa.fa_decode_cache(q, cache, table, n, o=given[0].transpose(1, 2)),
               lambda: fa.fa_decode_cache(q, cache, table, n, scale=-1.0),
               lambda: fa.fa_decode_cache(q, cache, table, n, workspace=ws[:100]),
               lambda: fa.fa_decode_cache(q, cache, table, n, pages=pages.long()),
               lambda: fa.fa_cache_select(q, cache, table, n, 2, 2, 1), lambda: fa.fa_cache_select(q, cache, table, n, 0),
               lambda: fa.fa_cache_select(q, cache._replace(k_mean=None, k_mean_scale=None), table, n, 5),
               lambda: fa.fa_cache_read(cache, table, n, -1), lambda: fa.fa_cache_read(cache, table, n, 5, torch.float32),
               lambda: fa.fa_cache_read(cache, table, n, 90, k=given[3][:3]),
               lambda: fa.fa_cache_write(cache, new, new[:3], table, n), lambda: fa.fa_cache_write(cache, new[:3], new[:3], table, n),
               lambda: fa.fa_cache_write(cache, new, new, table, n, cu_seqlens=n))
        said = []
        for call in bad:
            with pytest.raises(fa.FAError) as e:
                call()
            said.append(e.value.status)
        return out + list(given), said

    quick, quick_said = everything()
    monkeypatch.setattr(module, "_module", False)
    monkeypatch.setattr(module, "_bound", load())
    longer, longer_said = everything()
    assert not module._quick()
    assert quick_said == longer_said
    for x, y in zip(quick, longer):
        assert torch.equal(x.view(torch.uint8), y.view(torch.uint8))
    assert status(fa) == 0


def test_first_call_may_be_captured(fa):
    """A process whose first calls are inside a capture."""
    import subprocess
    import sys
    code = """
import sys, torch
sys.path[:0] = %r
import attention_forward_02_gb300 as fa
from cache_util import Ref, pages_for
table, pool = pages_for([70], 16, 1)
cache = Ref(pool, 1, 16, 32, "int8", 2).to("cuda")
table, lens = table.cuda(), torch.tensor([70], dtype=torch.int32, device="cuda")
q = torch.randn(1, 4, 1, 32, device="cuda").half()
x = torch.randn(1, 1, 32, device="cuda").half()
torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    fa.fa_cache_write(cache, x, x, table, lens)
    pages = fa.fa_cache_select(q, cache, table, lens, 3)
    o, lse = fa.fa_decode_cache(q, cache, table, lens, pages=pages)
    k, v = fa.fa_cache_read(cache, table, lens, 70)
g.replay()
torch.cuda.synchronize()
want = [t.clone() for t in (pages, o, lse, k, v)]
pages = fa.fa_cache_select(q, cache, table, lens, 3)
o, lse = fa.fa_decode_cache(q, cache, table, lens, pages=pages)
k, v = fa.fa_cache_read(cache, table, lens, 70)
assert all(torch.equal(a, b) for a, b in zip(want, (pages, o, lse, k, v)))
print("captured")
""" % ([p for p in sys.path if p][:8],)
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "captured" in r.stdout, r.stdout + r.stderr


def test_attention_strides_streams_and_outputs(fa):
    """Queries as a projection gives them, on a stream of their own, into given outputs."""
    lens = [70, 33]
    table, pool = pages_for(lens, 32, 1)
    ref = Ref(pool, 2, 32, 64, "e4m3", 2)
    qkv = randn((2, 3, 12, 64), torch.bfloat16, 3)
    q = qkv[:, :, 2:10].transpose(1, 2)
    cache, table_d, lens_d = ref.to("cuda"), dev(table), dev(lens)
    qd = qkv.cuda()[:, :, 2:10].transpose(1, 2)
    o = torch.empty((2, 8, 3, 64), dtype=torch.bfloat16, device="cuda")
    lse = torch.empty((2, 8, 3), device="cuda")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    # page numbers out of a wider table
    wide = torch.full((2, table.shape[1] + 5), -9, dtype=torch.int32, device="cuda")
    wide[:, 2:2 + table.shape[1]] = table_d
    s.wait_stream(torch.cuda.current_stream())
    got = fa.fa_decode_cache(qd, cache, wide[:, 2:2 + table.shape[1]], lens_d, causal=True, o=o, lse=lse, stream=s)
    s.synchronize()
    assert got[0] is o and got[1] is lse
    check_attention(fa, ref, q, table, lens, True, got=got)
    o2, none = fa.fa_decode_cache(qd, cache, table_d, lens_d, causal=True, return_lse=False)
    assert none is None and torch.equal(o2, o)


def test_large_cache_offsets(fa):
    """Codes beyond 2^32 bytes into a cache."""
    page, d, heads = 64, 128, 8
    pages = 2 ** 32 // (page * d * heads) + 40
    cache = fa.FACache.empty(pages, heads, page, d)
    small = Ref(5, heads, page, d, "e4m3", 2)
    lens = [150]
    table = torch.tensor([[pages - 1, 3, pages - 30]], dtype=torch.int32)
    new = [randn((150, heads, d), torch.bfloat16, s) for s in (3, 4)]
    fa.fa_cache_write(cache, new[0].cuda(), new[1].cuda(), dev(table), dev([0]))
    small.write(new[0], new[1], torch.tensor([[2, 3, 4]]), [0], [0, 150])
    for at, p in ((2, pages - 1), (3, 3), (4, pages - 30)):
        n = 150 - 128 if at == 4 else page
        assert same_values(cache.k[p, :, :n].float(), small.k[at, :, :n])
        assert same_values(cache.v_scale[p], small.v_scale[at])
    q = randn((1, 16, 1, d), torch.bfloat16, 5)
    got = fa.fa_decode_cache(q.cuda(), cache, dev(table), dev(lens))
    k, v = fa.fa_cache_read(cache, dev(table), dev(lens), 150)
    assert status(fa) == 0
    small_table = torch.tensor([[2, 3, 4]], dtype=torch.int32)
    check_attention(fa, small, q, small_table, lens, False, got=got)
    want = small.sequence(small_table[0], 150)
    assert same_values(k[0], want[0].bfloat16()) and same_values(v[0], want[1].bfloat16())


# ---------------------------------------------------------------------------
# selection


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("d,page", [(32, 16), (64, 32), (96, 64), (128, 16)])
@pytest.mark.parametrize("heads,G,Nq,slots,first,last", [(2, 1, 1, 3, 1, 1), (1, 8, 1, 12, 1, 1), (1, 3, 4, 7, 0, 2),
                                                         (1, 70, 2, 5, 2, 3), (2, 2, 1, 200, 1, 1)])
def test_select(fa, dtype, d, page, heads, G, Nq, slots, first, last):
    lens = [0, 3, page * slots, page * slots + 1, page * 150 + 5, page * 150]
    table, pool = pages_for(lens, page, 1)
    ref = Ref(pool, heads, page, d, "e4m3", 2)
    q = randn((len(lens), heads * G, Nq, d), DTYPES[dtype], 3)
    for causal in (False, True):
        got = fa.fa_cache_select(q.cuda(), ref.to("cuda"), dev(table), dev(lens), slots, keep_first=first,
                                 keep_last=last, causal=causal)
        assert status(fa) == 0
        want = ref.select(q, table, lens, slots, first, last, causal)
        assert torch.equal(got.cpu(), want)
        # the same out of a much wider table
        wide = torch.full((len(lens), 20000), -7, dtype=torch.int32)
        wide[:, :table.shape[1]] = table
        got = fa.fa_cache_select(q.cuda(), ref.to("cuda"), dev(wide), dev(lens), slots, keep_first=first,
                                 keep_last=last, causal=causal)
        assert status(fa) == 0
        assert torch.equal(got.cpu(), want)


@pytest.mark.parametrize("n,B,heads", [(9000, 1, 1), (3000, 40, 4), (700, 3, 64)])
def test_select_many_pages(fa, n, B, heads):
    """Thousands of pages (more than a block holds scores of, too), batches of many segments, equal scores."""
    page, d = 16, 32
    lens = [page * n - 3 * b for b in range(B)]
    ref = Ref(2000, heads, page, d, "e4m3", 2)
    ref.k_mean[:] = (ref.k_mean / 64).round()  # small whole numbers: many ties
    table = torch.randint(0, 2000, (B, n), generator=torch.Generator().manual_seed(4)).int()
    q = randn((B, heads, 1, d), torch.float16, 3)
    got = fa.fa_cache_select(q.cuda(), ref.to("cuda"), dev(table), dev(lens), 64).cpu()
    assert status(fa) == 0
    # a few of the lists against the definition, and all by their properties
    for b, h in ((0, 0), (B - 1, heads - 1), (B // 2, heads // 2)):
        s = [float(x) for x in _scores(ref, q[b, h, 0], table[b], h)][1:-(-lens[b] // page) - 1]
        best = sorted(range(len(s)), key=lambda j: (-s[j], j))[:62]
        assert got[b, h, 0].tolist() == sorted([0, -(-lens[b] // page) - 1] + [j + 1 for j in best])
    assert (got[..., 1:] > got[..., :-1]).all() and (got[..., 0] == 0).all()


@pytest.mark.parametrize("n", [255, 256, 257])
@pytest.mark.parametrize("slots,first,last", [(8, 1, 1), (254, 0, 1), (5, 3, 2)])
def test_select_table_widths(fa, n, slots, first, last):
    """Tables about the width where the number of threads changes, with ties and short sequences among them."""
    page, d, heads = 16, 64, 2
    lens = [page * n, page * n - 7, page * slots + 1, 0]
    ref = Ref(300, heads, page, d, "int8", 2)
    ref.k_mean[:] = (ref.k_mean / 32).round()
    table = torch.randint(0, 300, (len(lens), n), generator=torch.Generator().manual_seed(4)).int()
    q = randn((len(lens), heads, 2, d), torch.bfloat16, 3)
    got = fa.fa_cache_select(q.cuda(), ref.to("cuda"), dev(table), dev(lens), slots, keep_first=first, keep_last=last,
                             causal=True)
    assert status(fa) == 0
    assert torch.equal(got.cpu(), ref.select(q, table, lens, slots, first, last, True))


def _scores(ref, q, row, h):
    from cache_util import encode, finite_max, scale_of
    s = scale_of(finite_max(q.double()), 127.0)
    x = encode(q.double() / s, "int8")
    row = row.long()
    return (ref.k_mean[row, h] @ x) * s * ref.k_mean_scale[row, h]


def test_select_ties_and_special_queries(fa):
    """Equal scores go to the lower page; infinities in a query saturate, NaN counts as 0; a zero query."""
    page, d = 16, 32
    lens = [page * 600]
    table, pool = pages_for(lens, page, 1)
    ref = Ref(pool, 1, page, d, "e4m3", 2)
    ref.k_mean_scale[:] = 2.0 ** -6
    ref.k_mean[:] = ref.k_mean[:3].repeat(-(-pool // 3), 1, 1)[:pool]  # three kinds of page
    q = randn((1, 2, 1, d), torch.bfloat16, 3)
    for change in ("none", "zero", "special"):
        if change == "zero":
            q[0, :] = 0
        if change == "special":
            q = randn((1, 2, 1, d), torch.bfloat16, 4)
            q[0, 0, 0, 1], q[0, 0, 0, 2], q[0, 1, 0, 3] = math.inf, math.nan, -math.inf
        for slots in (2, 3, 250, 450, 599):
            got = fa.fa_cache_select(q.cuda(), ref.to("cuda"), dev(table), dev(lens), slots)
            assert torch.equal(got.cpu(), ref.select(q, table, lens, slots, 1, 1, False)), (change, slots)


def test_select_bad_pages(fa):
    """A page with a bad number scores lowest: it is chosen last."""
    page, d = 16, 32
    lens = [page * 8]
    ref = Ref(8, 1, page, d, "e4m3", 2)
    table = torch.tensor([[0, 1, 77, 2, -2, 3, 4, 5]], dtype=torch.int32)
    q = randn((1, 1, 1, d), torch.bfloat16, 3)
    for slots in (4, 6, 7):
        got = fa.fa_cache_select(q.cuda(), ref.to("cuda"), dev(table), dev(lens), slots)
        assert status(fa) == FA_ERR_BOUNDS
        assert torch.equal(got.cpu(), ref.select(q, table, lens, slots, 1, 1, False))


# ---------------------------------------------------------------------------
# together


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
def test_prompt_then_steps(fa, fmt):
    """A user's loop: prompts written, then steps that write a token, select pages and attend to them and to all."""
    page, d, heads, G = 16, 64, 2, 4
    lens = [100, 7, 49]
    steps = 20
    table, pool = pages_for([n + steps for n in lens], page, 1)
    ref = Ref(pool, heads, page, d, fmt, 2)
    cache = ref.to("cuda")
    table_d = dev(table)
    cu = [0, 100, 107, 156]
    k, v = (randn((156, heads, d), torch.bfloat16, s) for s in (3, 4))
    at = dev([0, 0, 0])
    fa.fa_cache_write(cache, k.cuda(), v.cuda(), table_d, at, cu_seqlens=dev(cu))
    ref.write(k, v, table, [0, 0, 0], cu)
    at += dev(lens)
    for step in range(steps):
        k, v = (randn((3, heads, d), torch.bfloat16, 10 + 3 * step + s, 1.0 + step / 4) for s in (0, 1))
        q = randn((3, heads * G, 1, d), torch.bfloat16, 500 + step)
        fa.fa_cache_write(cache, k.cuda(), v.cuda(), table_d, at)
        at += 1
        ref.write(k, v, table, [n + step for n in lens], [0, 1, 2, 3])
        now = [n + step + 1 for n in lens]
        pages = fa.fa_cache_select(q.cuda(), cache, table_d, at, 4)
        assert torch.equal(pages.cpu(), ref.select(q, table, now, 4, 1, 1, False))
        check_attention(fa, ref, q, table, now, False, pages=pages.cpu(),
                        got=fa.fa_decode_cache(q.cuda(), cache, table_d, at, pages=pages))
        check_attention(fa, ref, q, table, now, False, got=fa.fa_decode_cache(q.cuda(), cache, table_d, at))
    check_cache(cache, ref)
    # the cache read back is what fa_decode attends to
    k, v = fa.fa_cache_read(cache, table_d, at, max(now))
    o, _ = fa.fa_decode_cache(q.cuda(), cache, table_d, at)
    b = 0  # the longest sequence: no padding
    o16, _ = fa.fa_decode(q[b:b + 1].cuda().reshape(heads, 1, G, d).transpose(0, 1).contiguous(),
                          k[b:b + 1].contiguous(), v[b:b + 1].contiguous())
    assert (o16.reshape(-1).float() - o[b].reshape(-1).float()).abs().max() <= 2.0 ** -6 * o.abs().max()
    assert status(fa) == 0


def test_graph_replays_with_new_lengths(fa):
    """Captured steps read lengths, pages and tokens when they replay; two graphs with workspaces of their own."""
    page, d, heads = 16, 64, 2
    lens = [40, 3]
    table, pool = pages_for([n + 40 for n in lens], page, 1)
    ref = Ref(pool, heads, page, d, "e4m3", 2)
    cache = ref.to("cuda")
    table_d, at = dev(table), dev(lens)
    k, v = (torch.zeros(2, heads, d, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    q = torch.zeros(2, 8, 1, d, dtype=torch.bfloat16, device="cuda")

    def step():
        fa.fa_cache_write(cache, k, v, table_d, at)
        at.add_(1)
        pages = fa.fa_cache_select(q, cache, table_d, at, 3)
        return pages, fa.fa_decode_cache(q, cache, table_d, at), fa.fa_decode_cache(q, cache, table_d, at, pages=pages)

    graphs = []
    for _ in range(2):
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            step()
        torch.cuda.current_stream().wait_stream(side)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = step()
        graphs.append((g, out))
    # the warm-up steps wrote too: begin again
    for x, y in zip(cache, ref.to("cuda")):
        x.view(torch.uint8).copy_(y.view(torch.uint8))
    at.copy_(dev(lens))
    for i in range(20):
        new = [randn((2, heads, d), torch.bfloat16, 20 + i + 100 * s) for s in (0, 1)]
        qn = randn((2, 8, 1, d), torch.bfloat16, 300 + i)
        k.copy_(new[0]), v.copy_(new[1]), q.copy_(qn)
        g, (pages, dense, sparse) = graphs[i % 2]
        g.replay()
        ref.write(new[0], new[1], table, [n + i for n in lens], [0, 1, 2])
        now = [n + i + 1 for n in lens]
        assert torch.equal(pages.cpu(), ref.select(qn, table, now, 3, 1, 1, False))
        check_attention(fa, ref, qn, table, now, False, got=dense)
        check_attention(fa, ref, qn, table, now, False, pages=pages.cpu(), got=sparse)
    check_cache(cache, ref)
    assert status(fa) == 0


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
@pytest.mark.parametrize("d", [32, 64, 96, 128])
@pytest.mark.parametrize("G,Nq", [(1, 1), (16, 1), (4, 5)])
def test_checked_build(fa, monkeypatch, fmt, d, G, Nq):
    """The same calls through the library with device-side address checks."""
    from attention_forward_02_gb300 import _lib
    chk = _lib.load_checked()
    monkeypatch.setattr(_lib, "_lib", chk)
    page, heads, lens = 32, 2, [300, 1, 0, 77]
    table, pool = pages_for(lens, page, 1)
    ref = Ref(pool, heads, page, d, fmt, 2)
    cache = ref.to("cuda")
    k, v = (randn((378, heads, d), torch.bfloat16, s) for s in (3, 4))
    cu = [0, 300, 301, 301, 378]
    fa.fa_cache_write(cache, k.cuda(), v.cuda(), dev(table), dev([0] * 4), cu_seqlens=dev(cu))
    ref.write(k, v, table, [0] * 4, cu)
    check_cache(cache, ref)
    q = randn((4, heads * G, Nq, d), torch.bfloat16, 5)
    pages = fa.fa_cache_select(q.cuda(), cache, dev(table), dev(lens), 4, causal=True)
    assert torch.equal(pages.cpu(), ref.select(q, table, lens, 4, 1, 1, True))
    check_attention(fa, ref, q, table, lens, True)
    check_attention(fa, ref, q, table, lens, True, pages=pages.cpu())
    assert status(fa) == 0


def test_codes_are_what_torch_calls_them(fa):
    """A cache's buffers are plain torch tensors: values of a page by torch's own conversion."""
    for fmt in ("e4m3", "int8"):
        cache = fa.FACache.empty(2, 1, 16, 32, dtype=CODES[fmt])
        x = randn((16, 1, 32), torch.float16, 1)
        fa.fa_cache_write(cache, x.cuda(), x.cuda(), dev([[1]]), dev([0]))
        back = cache.k[1, 0].float() * cache.k_scale[1, 0]
        step = 2.0 ** -4 * x[:, 0].abs().float() + 2.0 ** -8 if fmt == "e4m3" else float(cache.k_scale[1, 0]) / 2
        assert ((back.cpu() - x[:, 0].float()).abs() <= step).all()
