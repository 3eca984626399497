"""fa_rope in place on query and key rows whose elements lie between one another's: disjoint views are taken, views
with an element in common refused.  Fake addresses: without a GPU a call that is taken gets as far as CUDA (status 4)."""
import ctypes
import itertools
import random

import pytest
import torch

import attention_forward_02_gb300 as fa
from attention_forward_02_gb300.build import build_library

BASE, TURNS = 0x10000000, 0x50000000

pytestmark = pytest.mark.skipif(torch.cuda.is_available(), reason="fake addresses would reach the GPU")


@pytest.fixture(scope="module", autouse=True)
def lib():
    build_library()
    return fa.load()


def call(q, k, q_out=None, k_out=None, B=1, N=1, d=64):
    """Views are (first element, batch stride, head stride, row stride, heads)."""
    rope = fa.RopeDesc(TURNS, 16, 0, 1.0)
    rows = []
    for x, y in ((q, q_out or q), (k, k_out or k)):
        rows.append(fa.RopeRows(BASE + 2 * x[0], BASE + 2 * y[0], *x[1:4], *y[1:4], x[4]))
    return fa.fa_rope_raw(ctypes.byref(rope), ctypes.byref(rows[0]), ctypes.byref(rows[1]), None, 0, B, N, d, 0, 0, None)


@pytest.mark.parametrize("H,N,d", [(8, 5, 64), (1, 7, 64), (3, 1, 128), (40, 4096, 128)])
def test_a_head_s_query_key_and_value_side_by_side(H, N, d):
    """[T, H, 3, d] and [B, N, H, 3, d]."""
    row = H * 3 * d
    q, k, v = ((i * d, N * row, 3 * d, row, H) for i in range(3))
    for B in (1, 2, 6):
        assert call(q, k, B=B, N=N, d=d) == 4
        assert call(k, v, B=B, N=N, d=d) == 4
        assert call(q, q, B=B, N=N, d=d) == 1
        half = (d // 2, *k[1:])  # half of the queries' channels, half of the keys'
        assert call(q, half, B=B, N=N, d=d) == 1
    # out of place into the value's and the key's places, and onto one another
    assert call(q, k, v, k, B=2, N=N, d=d) == 4
    assert call(q, k, k, q, B=2, N=N, d=d) == 1


@pytest.mark.parametrize("B,Hq,H,N,d", [(2, 8, 2, 5, 64), (3, 4, 4, 1, 32), (2, 32, 8, 2048, 128)])
def test_heads_of_every_batch(B, Hq, H, N, d):
    """[B, Hq + H, N, d] cut along the heads."""
    batch = (Hq + H) * N * d
    q, k = (0, batch, N * d, d, Hq), (Hq * N * d, batch, N * d, d, H)
    assert call(q, k, B=B, N=N, d=d) == 4
    assert call(q, ((Hq - 1) * N * d, *k[1:]), B=B, N=N, d=d) == 1
    assert call(q, k[:4] + (H + 1,), B=B, N=N, d=d) == 1   # the last head is the next batch's first


def elements(view, B, N, d):
    at, batch, head, row, heads = view
    return [at + b * batch + h * head + n * row + c
            for b, h, n, c in itertools.product(range(B), range(heads), range(N), range(0, d, 8))]


@pytest.mark.parametrize("seed", range(8))
def test_views_of_one_buffer(seed):
    """Slices of a contiguous buffer's dimensions, in any order, against their sets of elements."""
    rng = random.Random(seed)
    d, taken, refused = 32, 0, 0
    for _ in range(400):
        sizes = [rng.randint(1, 4) for _ in range(4)]
        strides = [0] * 4
        step = d
        for i in reversed(range(4)):
            strides[i], step = step, step * sizes[i]
        dims = rng.sample(range(4), 3)
        extent = [rng.randint(1, sizes[x]) for x in dims]
        views = []
        for which in range(2):
            own = extent if which == 0 or rng.random() < 0.5 else extent[:2] + [rng.randint(1, sizes[dims[2]])]
            at = sum(strides[x] * rng.randint(0, sizes[x] - (own[dims.index(x)] if x in dims else 1)) for x in range(4))
            at += rng.choice([0, 0, 0, 8])
            views.append((at, strides[dims[0]], strides[dims[2]], strides[dims[1]], own[2]))
        B, N = extent[:2]
        q, k = (elements(v, B, N, d) for v in views)
        common = bool(set(q) & set(k))
        assert call(*views, B=B, N=N, d=d) == (1 if common else 4), (views, B, N)
        taken, refused = taken + (not common), refused + common
    assert taken > 50 and refused > 50
