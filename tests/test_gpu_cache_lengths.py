"""Lengths on the device that no page table holds: reported, and never written for."""
import pytest
import torch

from cache_util import DTYPES, Ref

pytestmark = pytest.mark.gpu

FA_ERR_BOUNDS = 6
PAGE, D, HEADS = 16, 64, 2
TABLE = [[0, 1, 2], [3, 4, 5], [6, 7, 8], [9, 10, 11]]


@pytest.fixture
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


def randn(shape, dtype, seed):
    return torch.randn(shape, generator=torch.Generator().manual_seed(seed)).to(dtype).cuda()


def wide(columns):
    """The table with more places, which hold a page of nobody."""
    t = torch.full((4, columns), 12, dtype=torch.int32)
    t[:, :3] = torch.tensor(TABLE, dtype=torch.int32)
    return t.cuda()


# what a call reads, and whether it has to be reported
LENGTHS = [([48, 0, 17, 1], False), ([48, 49, 17, 1], True), ([2 ** 31 - 1, 0, 0, 0], True), ([48, 0, 17, -1], True),
           ([-2 ** 31, 3, 3, 3], True)]


@pytest.mark.parametrize("lens,bad", LENGTHS)
def test_reading_calls_report_lengths(fa, lens, bad):
    """All page numbers are good here, so that the lengths alone are at issue; the results are those of the lengths cut
    to the table."""
    cache = Ref(13, HEADS, PAGE, D, "e4m3", 2).to("cuda")
    q = randn((4, 4, 1, D), torch.bfloat16, 3)
    cut = dev([min(max(n, 0), 48) for n in lens])
    lens, table = dev(lens), dev(TABLE)
    calls = [lambda n: fa.fa_decode_cache(q, cache, table, n), lambda n: fa.fa_cache_read(cache, table, n, 60),
             lambda n: (fa.fa_cache_select(q, cache, table, n, 2),), lambda n: (fa.fa_cache_select(q, cache, table, n, 3),)]
    pages = fa.fa_cache_select(q, cache, table, cut, 2)
    calls.append(lambda n: fa.fa_decode_cache(q, cache, table, n, pages=pages))
    for call in calls:
        want = call(cut)
        assert status(fa) == 0
        got = call(lens)
        assert status(fa) == (FA_ERR_BOUNDS if bad else 0)
        assert all(torch.equal(x, y) for x, y in zip(got, want))


@pytest.mark.parametrize("over", [0, 1])
def test_a_shared_out_call_reports_lengths(fa, over):
    """Contexts of many units, and more sequences than threads of a block."""
    B, columns = 300, 400
    cache = Ref(13, HEADS, PAGE, D, "int8", 2).to("cuda")
    table = torch.zeros(B, columns, dtype=torch.int32, device="cuda")
    lens = torch.full((B,), 20, dtype=torch.int32)
    lens[7] = columns * PAGE
    q = randn((B, 2, 1, D), torch.float16, 3)
    fa.fa_decode_cache(q, cache, table, lens.cuda())
    assert status(fa) == 0
    lens[257] = columns * PAGE + 1 if over else -3
    fa.fa_decode_cache(q, cache, table, lens.cuda())
    assert status(fa) == FA_ERR_BOUNDS


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("rows", [1, 5, 40])  # by steps (no more rows than sequences), and by pages
def test_a_negative_length_is_not_written_for(fa, fmt, dtype, rows):
    ref = Ref(13, HEADS, PAGE, D, fmt, 2)
    before = [-1, 5, -2 ** 31, 0] if rows > 1 else [7, -1, -2 ** 31, 0]
    cache, want = ref.to("cuda"), ref.to("cuda")
    k, v = (randn((4 * rows, HEADS, D), DTYPES[dtype], s) for s in (3, 4))
    table = wide(4)
    fa.fa_cache_write(cache, k, v, table, dev(before))
    assert status(fa) == FA_ERR_BOUNDS
    # the others are written as without them
    cu, n = [0], 0
    for b in before:
        n += rows if b >= 0 else 0
        cu.append(n)
    keep = torch.cat([torch.arange(i * rows, (i + 1) * rows) for i, b in enumerate(before) if b >= 0]).cuda()
    fa.fa_cache_write(want, k[keep], v[keep], table, dev(before), cu_seqlens=dev(cu))
    assert status(fa) == 0  # a negative length of a sequence without new rows harms nothing
    for x, y in zip(cache, want):
        assert torch.equal(x.view(torch.uint8), y.view(torch.uint8))
    # and alone
    cache = ref.to("cuda")
    fa.fa_cache_write(cache, k[:rows], v[:rows], table[:1], dev([-3]))
    assert status(fa) == FA_ERR_BOUNDS
    for x, y in zip(cache, ref.to("cuda")):
        assert torch.equal(x.view(torch.uint8), y.view(torch.uint8))
