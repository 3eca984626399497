"""Strides whose span leaves 64 bits: refused by every call over the paged caches before any sum of them (a wrapped one
would let an output lie over an input).  Fake addresses: no call gets as far as CUDA."""
import ctypes

import pytest

import attention_forward_02_gb300 as fa
from attention_forward_02_gb300.build import build_library

A = [0x1000000000 * (i + 1) for i in range(14)]
HUGE = [1 << 41, 1 << 61, (1 << 62) + 8, (1 << 63) - 8]


@pytest.fixture(scope="module", autouse=True)
def lib():
    build_library()
    return fa.load()


def cache4():
    return ctypes.byref(fa.Cache4Desc(A[0], 10, 2, 16, 64))


def cache8():
    return ctypes.byref(fa.CacheDesc(*A[:6], 10, 2, 16, 64, 0))


@pytest.mark.parametrize("huge", HUGE)
@pytest.mark.parametrize("place", range(4))
def test_rows_that_are_written(huge, place):
    s = [128, 64, 128, 64]
    s[place] = huge
    assert fa.fa_cache4_write_raw(cache4(), A[6], A[7], *s, A[8], 5, 0, None) == 1
    assert fa.fa_cache_write_raw(cache8(), A[6], A[7], *s, None, A[8], A[9], 4, 4, 5, 5, 0, None) == 1


@pytest.mark.parametrize("huge", HUGE)
@pytest.mark.parametrize("place", range(4))
def test_queries_and_tables(huge, place):
    s, stride = [512, 64, 256], 4
    if place == 3:
        stride = huge
    else:
        s[place] = huge
    B, Hq, Nq = 3, 8, 2
    assert fa.fa_decode_cache4_raw(cache4(), A[6], *s, A[7], A[8], A[9], A[10], stride, 4, A[11], 1 << 34, B, Hq, Nq, 0.1, 0, 0,
                                   None) == 1
    assert fa.fa_decode_cache_raw(cache8(), A[6], *s, A[7], A[8], A[9], A[10], stride, 4, None, 0, A[11], 1 << 34, B, Hq, Nq,
                                  0.1, 0, 0, None) == 1
    assert fa.fa_cache_select_raw(cache8(), A[6], *s, A[9], A[10], stride, 4, A[7], 4, 1, 1, A[11], 1 << 34, B, Hq, Nq, 0, 0,
                                  None) == 1


@pytest.mark.parametrize("huge", HUGE)
def test_tables(huge):
    assert fa.fa_cache4_read_raw(cache4(), A[6], A[7], A[8], A[9], huge, 4, 3, 20, 0, None) == 1
    assert fa.fa_cache_read_raw(cache8(), A[6], A[7], A[8], A[9], huge, 4, 3, 20, 0, None) == 1
    assert fa.fa_cache_plan_raw(A[0], 10, A[1], A[2], huge, 4, A[3], A[4], A[5], A[6], A[7], A[8], A[1], 16, 3, 9, None) == 1
    assert fa.fa_cache_trim_raw(A[0], 10, A[1], A[2], huge, 4, A[3], A[4], A[1], 16, 3, None) == 1
