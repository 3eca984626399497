"""Attention over the 8-bit cache on the GPU within bounds that each row's own keys and weights give (cache_bounds;
test_cache_bounds_cpu.py shows that a wrong tile of V exceeds them)."""
import pytest
import torch

from cache_bounds import attend_bounds, excess, tiles_apart
from cache_util import DTYPES, Ref, pages_for

pytestmark = pytest.mark.gpu


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
    return (torch.randn(shape, generator=torch.Generator().manual_seed(seed)) * scale).to(dtype)


def check(fa, ref, q, table, lens, causal=False, pages=None):
    scale = q.shape[-1] ** -0.5
    o, lse = fa.fa_decode_cache(q.cuda(), ref.to("cuda"), dev(table), dev(lens), causal=causal,
                                pages=None if pages is None else dev(pages))
    assert status(fa) == 0
    o, lse = o.double().cpu(), lse.double().cpu()
    want = attend_bounds(ref, q, table, lens, scale, causal, pages)
    empty = torch.isinf(want[1])
    assert torch.equal(empty, torch.isinf(lse) & (lse < 0)) and not o[empty].any()
    over, lse_over = excess(o, lse, want)
    assert over <= 0 and lse_over <= 0, "o %.3g, lse %.3g of its bound over it" % (over, lse_over)


# rows of a KV head: one to eight, two row groups of a warp, two and four warps along the rows, several groups
ROWS = [(1, 1), (4, 1), (4, 3), (16, 1), (6, 5), (16, 4), (10, 16)]


@pytest.mark.parametrize("d", [32, 64, 96, 128])
@pytest.mark.parametrize("G,Nq", ROWS)
def test_long_sequences(fa, d, G, Nq):
    """Long sequences beside short ones: parts of one sequence in many blocks, many sequences in one."""
    lens = [6000, 3, 1, 1500, 0, 64, 65] if G * Nq <= 4 else [2500, 3, 700]
    table, pool = pages_for(lens, 64, 1)
    ref = tiles_apart(Ref(pool, 1, 64, d, "e4m3", 2))
    ref.v_scale[:] = 2.0 ** -5
    check(fa, ref, randn((len(lens), G, Nq, d), torch.float16, 3), table, lens, True)


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("page", [16, 32, 64, 128])
@pytest.mark.parametrize("d,heads,G", [(32, 1, 16), (64, 2, 4), (96, 1, 3), (128, 2, 8)])
def test_short_sequences(fa, fmt, dtype, page, d, heads, G):
    """A block a sequence."""
    lens = [1, 0, 16, 17, 129, 300, 500]
    table, pool = pages_for(lens, page, 1)
    ref = tiles_apart(Ref(pool, heads, page, d, fmt, 2))
    check(fa, ref, randn((len(lens), heads * G, 2, d), DTYPES[dtype], 3), table, lens, True)


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
@pytest.mark.parametrize("G", [1, 8, 20])
def test_uneven_scales(fa, fmt, G):
    """Pages whose V scales double (or halve) from each to the next."""
    lens = [640, 640]
    table, pool = pages_for(lens, 16, 1)
    ref = tiles_apart(Ref(pool, 2, 16, 64, fmt, 2))
    for b, sign in ((0, 1), (1, -1)):
        for at in range(40):
            p = int(table[b, at])
            ref.v_scale[p] = 2.0 ** (sign * (at - 20))
            ref.k_scale[p] = 2.0 ** (-10 + at // 6)
    check(fa, ref, randn((2, 2 * G, 1, 64), torch.bfloat16, 3), table, lens)


@pytest.mark.parametrize("page", [16, 64])
@pytest.mark.parametrize("G", [4, 12])
def test_scales_that_are_no_powers_of_two(fa, page, G):
    lens = [1333, 64]
    table, pool = pages_for(lens, page, 1)
    ref = tiles_apart(Ref(pool, 2, page, 128, "int8", 2))
    g = torch.Generator().manual_seed(9)
    ref.k_scale, ref.v_scale = (torch.rand(ref.k_scale.shape, generator=g).float().double() * 0.03 + 0.01 for _ in range(2))
    check(fa, ref, randn((2, 2 * G, 1, 128), torch.float16, 3), table, lens)


@pytest.mark.parametrize("d", [32, 128])
@pytest.mark.parametrize("G", [3, 12])
def test_listed_pages(fa, d, G):
    """Lists that go to many blocks, beside a sequence that has fewer pages than slots."""
    page, lens = 32, [6000, 500]
    table, pool = pages_for(lens, page, 1)
    ref = tiles_apart(Ref(pool, 2, page, d, "e4m3", 2))
    g = torch.Generator().manual_seed(5)
    pages = torch.full((2, 2, 2, 120), -1, dtype=torch.int32)
    for h in range(2):
        for i in range(2):
            pages[0, h, i] = torch.randperm(6000 // page, generator=g)[:120].int()
            pages[1, h, i, :16] = torch.arange(16)
    check(fa, ref, randn((2, 2 * G, 2, d), torch.float16, 3), table, lens, False, pages)


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
def test_peaked_and_rising_scores(fa, fmt):
    """Scores that spread over hundreds, and scores that rise along the keys, so that the reference moves."""
    lens = [900, 900]
    table, pool = pages_for(lens, 64, 1)
    ref = tiles_apart(Ref(pool, 1, 64, 128, fmt, 2))
    q = randn((2, 8, 1, 128), torch.float16, 3)
    check(fa, ref, q * 8, table, lens)
    for at in range(15):
        p = int(table[1, at])
        ref.k[p] = ref.k[p].abs()
        ref.k_scale[p] = 2.0 ** -9 * (1 if at < 5 else 2 if at < 10 else 4)
    check(fa, ref, q.abs() * 4, table, lens)


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
@pytest.mark.parametrize("G", [4, 20])
@pytest.mark.parametrize("low,high", [(-80, -80), (100, 100), (-60, 40), (-80, 20)])
def test_scales_at_the_ends_of_their_range(fa, fmt, G, low, high):
    """V scales as small and as large as they may be, and as far apart within one sequence; small and large ones take
    turns, so that half of the weight is at pages of the lowest."""
    page, n = 16, 700
    table, pool = pages_for([n], page, 1)
    ref = tiles_apart(Ref(pool, 1, page, 64, fmt, 2))
    for at in range(-(-n // page)):
        ref.v_scale[int(table[0, at])] = 2.0 ** (low if at % 2 else high)
    check(fa, ref, randn((1, G, 1, 64), torch.bfloat16, 3), table, [n])
