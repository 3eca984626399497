"""The bounds that attention over the 8-bit cache is held to find a wrong tile of V: small faults are planted in the
64-bit definition and have to exceed them."""
import copy
import math

import pytest
import torch

from cache_bounds import attend_bounds, excess, tiles_apart
from cache_util import Ref, pages_for


def randn(shape, dtype, seed):
    return torch.randn(shape, generator=torch.Generator().manual_seed(seed)).to(dtype)


def long_case(d):
    lens = [6000]
    table, pool = pages_for(lens, 64, 1)
    ref = tiles_apart(Ref(pool, 1, 64, d, "e4m3", 2))
    ref.v_scale[:] = 2.0 ** -5
    return ref, randn((1, 4, 1, d), torch.float16, 3), table, lens


def uneven_case(fmt, sign):
    """Pages whose V scales double (or halve) from each to the next, as in the GPU's test."""
    lens = [640]
    table, pool = pages_for(lens, 16, 1)
    ref = tiles_apart(Ref(pool, 2, 16, 64, fmt, 2))
    for at in range(40):
        p = int(table[0, at])
        ref.v_scale[p] = 2.0 ** (sign * (at - 20))
        ref.k_scale[p] = 2.0 ** (-10 + at // 6)
    return ref, randn((1, 8, 1, 64), torch.bfloat16, 3), table, lens


def tile(ref, table, n):
    """Page and slots of the n-th tile of 16 keys."""
    p, at = int(table[0, n * 16 // ref.page]), n * 16 % ref.page
    return p, slice(at, at + 16)


def plant(ref, table, n, fault):
    bad = copy.deepcopy(ref)
    p, rows = tile(ref, table, n)
    if fault == "zeroed":
        bad.v[p, :, rows] = 0
    elif fault == "doubled":
        bad.v[p, :, rows] *= 2
    else:  # as a stage or page taken for the one beside it gives (two swapped ones would cancel at equal weights)
        o, other = tile(ref, table, n - 1 if n else 1)
        bad.v[p, :, rows] = ref.v[o, :, other] * (ref.v_scale[o] / ref.v_scale[p])[:, None, None]
    return bad


@pytest.mark.parametrize("fault", ["zeroed", "doubled", "neighbour's"])
@pytest.mark.parametrize("d", [32, 128])
def test_planted_faults_in_a_long_sequence(d, fault):
    """One tile of 375."""
    ref, q, table, lens = long_case(d)
    want = attend_bounds(ref, q, table, lens, d ** -0.5, False)
    assert (want[2] > 0).all()
    for n in [*range(6), *range(180, 190), *range(370, 375)]:
        o, lse, _, _ = attend_bounds(plant(ref, table, n, fault), q, table, lens, d ** -0.5, False)
        assert torch.equal(lse, want[1])
        assert excess(o, lse, want)[0] > 0, n


@pytest.mark.parametrize("fault", ["zeroed", "doubled", "neighbour's"])
@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
@pytest.mark.parametrize("sign,tiles", [(1, [39, 38, 37, 36, 35]), (-1, [0, 1, 2, 3, 4])])
def test_planted_faults_among_uneven_scales(fmt, sign, tiles, fault):
    """The pages with the five largest of the scales."""
    ref, q, table, lens = uneven_case(fmt, sign)
    want = attend_bounds(ref, q, table, lens, 0.125, False)
    for n in tiles:
        o, lse, _, _ = attend_bounds(plant(ref, table, n, fault), q, table, lens, 0.125, False)
        assert excess(o, lse, want)[0] > 0, n


def test_bounds_by_hand():
    """One key: o is its value, with the roundings of P (1, exact) and of o; and a bound that is a rounding wide."""
    ref = Ref(1, 1, 16, 32, "int8", 2)
    ref.k[0, 0, 0], ref.v[0, 0, 0], ref.v_scale[0, 0] = 1.0, 100.0, 0.5
    ref.k_scale[0, 0] = 2.0 ** -5
    q = torch.ones(1, 1, 1, 32, dtype=torch.float16)
    o, lse, bo, bl = attend_bounds(ref, q, torch.zeros(1, 1, dtype=torch.int32), [1], 1.0, False)
    assert (o == 50.0).all() and float(lse) == 1.0  # 32 codes of 1
    assert 50 * 2.0 ** -11 < float(bo.max()) < 50 * 2.0 ** -10 and float(bl) < 2.0 ** -14
    assert excess(o + bo, lse, (o, lse, bo, bl)) == pytest.approx((0.0, -1.0), abs=1e-6)
    assert excess(o, lse + 2 * bl, (o, lse, bo, bl)) == pytest.approx((-1.0, 1.0), abs=1e-6)
    assert math.isnan(excess(o * math.nan, lse, (o, lse, bo, bl))[0])  # which no comparison passes
