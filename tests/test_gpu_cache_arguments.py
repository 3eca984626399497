"""Arguments of the 8-bit cache's Python functions that the C ABI cannot see: whole numbers that 32 bits do not hold,
and a selection without query heads.  Through the CPython module and through ctypes."""
import pytest
import torch

from cache_util import Ref

pytestmark = pytest.mark.gpu

HUGE = 2 ** 32


@pytest.fixture(params=["module", "ctypes"])
def fa(request, monkeypatch):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import attention_forward_02_gb300 as fa
    from attention_forward_02_gb300 import cache
    if request.param == "ctypes":
        monkeypatch.setattr(cache, "_module", False)
        monkeypatch.setattr(cache, "_bound", fa.load())
    assert bool(cache._quick()) == (request.param == "module")
    return fa


def case():
    cache = Ref(9, 2, 16, 32, "e4m3", 2).to("cuda")
    table = torch.arange(9, dtype=torch.int32, device="cuda")[None]
    q = torch.ones(1, 4, 1, 32, dtype=torch.float16, device="cuda")
    return cache, table, torch.tensor([140], dtype=torch.int32, device="cuda"), q


@pytest.mark.parametrize("kw", [dict(keep_first=HUGE), dict(keep_first=HUGE + 1), dict(keep_last=HUGE + 1),
                                dict(keep_first=1 - HUGE), dict(keep_last=2 ** 31), dict(slots=HUGE + 4),
                                dict(slots=2 ** 31)], ids=str)
def test_select_refuses_numbers_beyond_32_bits(fa, kw):
    cache, table, lens, q = case()
    given = torch.full((1, 2, 1, 4), -9, dtype=torch.int32, device="cuda")
    with pytest.raises(fa.FAError) as e:
        fa.fa_cache_select(q, cache, table, lens, **{"slots": 4, "pages": given, **kw})
    assert e.value.status == 1
    assert (given == -9).all()


def test_select_does_not_allocate_for_slots_beyond_32_bits(fa):
    cache, table, lens, q = case()
    torch.cuda.reset_peak_memory_stats()
    with pytest.raises(fa.FAError):
        fa.fa_cache_select(q, cache, table, lens, HUGE + 4)
    assert torch.cuda.max_memory_allocated() < 1 << 30


def test_read_refuses_lengths_beyond_32_bits(fa):
    cache, table, lens, _ = case()
    with pytest.raises(fa.FAError) as e:
        fa.fa_cache_read(cache, table, lens, HUGE + 3)
    assert e.value.status == 1


def test_write_refuses_rows_beyond_32_bits(fa):
    cache, table, lens, _ = case()
    before = [x.clone() for x in cache]
    x = torch.ones(1, 2, 32, dtype=torch.float16, device="cuda").expand(HUGE + 1, 2, 32)
    with pytest.raises(fa.FAError) as e:
        fa.fa_cache_write(cache, x, x, table, lens)
    assert e.value.status == 1
    torch.cuda.synchronize()
    assert all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip(cache, before))


def test_select_refuses_heads_beyond_32_bits(fa):
    """Rows that are all one row, by a stride of zero: four heads are left of them in 32 bits."""
    cache, table, lens, q = case()
    with pytest.raises(fa.FAError) as e:
        fa.fa_cache_select(q[:, :1].expand(1, HUGE + 4, 1, 32), cache, table, lens, 4)
    assert e.value.status == 1


def test_select_without_query_heads(fa):
    """Its output would not be empty, and nothing says what it holds."""
    cache, table, lens, q = case()
    for pages in (None, torch.full((1, 2, 1, 4), -9, dtype=torch.int32, device="cuda")):
        with pytest.raises(fa.FAError) as e:
            fa.fa_cache_select(q[:, :0], cache, table, lens, 4, pages=pages)
        assert e.value.status == 1
    assert (pages == -9).all()
    # attention without query heads has an empty result
    o, lse = fa.fa_decode_cache(q[:, :0], cache, table, lens)
    assert o.shape == (1, 0, 1, 32) and lse.shape == (1, 0, 1)
    # and so has a selection for no sequences
    assert fa.fa_cache_select(q[:0], cache, table[:0], lens[:0], 4).shape == (0, 2, 1, 4)
