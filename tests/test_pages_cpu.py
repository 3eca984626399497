"""fa_cache_plan and fa_cache_trim: what they refuse before any CUDA call, and the definition that the GPU tests use."""
import pytest
import torch

import attention_forward_02_gb300 as fa
import pages_util
from attention_forward_02_gb300.build import build_library

RING, COUNTS, TABLE, LENS, NEW, CU, ENDS, POS, SLOTS, OUT = (0x10000000 + i * 0x1000000 for i in range(10))


@pytest.fixture(scope="module", autouse=True)
def lib():
    build_library()
    return fa.load()


def plan(ring=RING, num_pages=100, counts=COUNTS, table=TABLE, stride=8, P=8, lens=LENS, new=NEW, cu=CU, ends=ENDS,
         pos=POS, slots=SLOTS, out=COUNTS, page=16, B=4, T=64):
    return fa.fa_cache_plan_raw(ring, num_pages, counts, table, stride, P, lens, new, cu, ends, pos, slots, out, page, B, T,
                                None)


def trim(ring=RING, num_pages=100, counts=COUNTS, table=TABLE, stride=8, P=8, lens=LENS, keep=NEW, out=COUNTS, page=16,
         B=4):
    return fa.fa_cache_trim_raw(ring, num_pages, counts, table, stride, P, lens, keep, out, page, B, None)


BOTH = [(dict(page=48), 2), (dict(page=8), 2), (dict(B=16385), 2), (dict(num_pages=1 << 27), 2), (dict(P=1 << 27, stride=1 << 27), 2),
        (dict(num_pages=0), 1), (dict(P=0), 1), (dict(stride=7), 1), (dict(B=-1), 1),
        (dict(ring=0), 1), (dict(counts=0), 1), (dict(table=0), 1), (dict(lens=0), 1), (dict(out=0), 1),
        (dict(ring=RING + 2), 3), (dict(counts=COUNTS + 4), 3), (dict(table=TABLE + 1), 3), (dict(lens=LENS + 2), 3),
        (dict(out=OUT + 4), 3), (dict(out=COUNTS + 8), 1), (dict(out=RING), 1), (dict(out=TABLE), 1), (dict(out=LENS), 1),
        (dict(B=0, ring=0), 0)]


@pytest.mark.parametrize("kwargs,status", BOTH + [
    (dict(T=-1), 1), (dict(new=0), 1), (dict(cu=0), 1), (dict(ends=0), 1), (dict(pos=0), 1), (dict(slots=0), 1),
    (dict(new=NEW + 2), 3), (dict(cu=CU + 1), 3), (dict(ends=ENDS + 2), 3), (dict(pos=POS + 2), 3), (dict(slots=SLOTS + 2), 3),
    (dict(ends=LENS), 1), (dict(cu=LENS + 12), 1), (dict(cu=NEW), 1), (dict(pos=TABLE), 1), (dict(slots=POS + 4), 1),
    (dict(ends=CU + 16), 1), (dict(slots=RING + 396), 1), (dict(pos=OUT, out=OUT + 8), 1), (dict(table=RING), 1),
], ids=str)
def test_plan_refusals(kwargs, status):
    assert plan(**kwargs) == status


@pytest.mark.parametrize("kwargs,status", BOTH + [(dict(keep=0), 1), (dict(keep=NEW + 2), 3), (dict(ring=TABLE), 1),
                                                  (dict(ring=LENS), 1), (dict(ring=NEW), 1), (dict(ring=COUNTS), 1)], ids=str)
def test_trim_refusals(kwargs, status):
    assert trim(**kwargs) == status


def test_python_refusals():
    pool = fa.FAPagePool.full(10, device="cpu")
    t, n = torch.zeros(2, 4, dtype=torch.int32), torch.zeros(2, dtype=torch.int32)
    for f in (lambda: fa.fa_cache_plan(pool, t, n, n, 16, 4), lambda: fa.fa_cache_trim(pool, t, n, n, 16),
              lambda: fa.fa_cache_plan((pool.ring, pool.counts), t, n, n, 16, 4)):
        with pytest.raises(fa.FAError) as e:
            f()
        assert e.value.status == 1


def test_definition():
    """By hand: two pages of 4 tokens held, three free, the ring gone round."""
    ring, counts, table = [7, 1, 9, -5, -5], [10, 13], [[4, 3, -1], [2, -1, -1], [-1, -1, -1]]
    got = pages_util.plan(ring, counts, table, [5, 4, 0], [4, 1, 9], 4, 14)
    assert got[0] == [[4, 3, 7], [2, 1, -1], [-1, -1, -1]]
    assert got[1:4] == ([0, 4, 5, 14], [9, 5, 0], [5, 6, 7, 8, 4] + [-1] * 9)
    # page 7 is none of the five: row 3 has no slot, which is reported
    assert got[4:] == ([13, 14, 15, -1, 4] + [-1] * 9, [12, 13], True)
    # sequence 0 gives page 7 back, sequence 1 pages 2 and 1, behind place 13 of the ring
    assert pages_util.trim(ring, [12, 13], got[0], [9, 5, 0], [5, 0, 0], 4) == ([1, 1, 9, 7, 2], [12, 16], True)
