"""Refusals of the 8-bit paged cache's entry points: before any CUDA call in C,
with fake addresses, and on the Python side with CPU tensors.  And the 64-bit
definition that the GPU tests compare with, pinned by hand."""
import ctypes
import math

import pytest
import torch

import attention_forward_02_gb300 as fa
from attention_forward_02_gb300 import _lib
from attention_forward_02_gb300.build import build_library
from cache_util import Ref, encode, scale_of


@pytest.fixture(scope="module", autouse=True)
def lib():
    build_library()
    return fa.load()


# well-separated, aligned fake addresses
K, V, KS, VS, M, MS = (0x100000000 * (i + 1) for i in range(6))
Q, O, L, W, LENS, TABLE, CU, PAGES, KN, VN = (0x1000000000 * (i + 1) for i in range(10))


def desc(**kw):
    a = dict(k=K, v=V, k_scale=KS, v_scale=VS, k_mean=M, k_mean_scale=MS, num_pages=100, heads=2, page=32, d=64,
             format=0)
    a.update(kw)
    return _lib.CacheDesc(**a)


BAD_CACHES = [(dict(c=c), status) for c, status in [
    (dict(k=0), 1), (dict(v_scale=0), 1), (dict(k_mean=0), 1), (dict(k_mean_scale=0), 1), (dict(num_pages=0), 1),
    (dict(heads=0), 1), (dict(page=48), 2), (dict(page=256), 2), (dict(page=8), 2), (dict(d=48), 2), (dict(d=256), 2),
    (dict(format=2), 2), (dict(heads=40000), 2), (dict(k=K + 8), 3), (dict(k_mean=M + 4), 3), (dict(v_scale=VS + 2), 3),
    (dict(v=K + 4096), 1), (dict(k_scale=VS + 16), 1),
]]


def write(c={}, k=KN, v=VN, strides=(128, 64, 128, 64), cu=CU, lens=LENS, table=TABLE, table_stride=9, P=9, B=3,
          T=10, dtype=1):
    return fa.fa_cache_write_raw(ctypes.byref(desc(**c)), k, v, *strides, cu, lens, table, table_stride, P, B,
                                 T, dtype, None)


@pytest.mark.parametrize("kw,status", BAD_CACHES + [
    (dict(dtype=2), 2), (dict(B=-1), 1), (dict(T=-1), 1), (dict(B=70000), 2), (dict(lens=0), 1),
    (dict(table=0), 1), (dict(P=0), 1), (dict(table_stride=8), 1), (dict(P=1 << 30, table_stride=1 << 30), 2),
    (dict(lens=LENS + 2), 3), (dict(cu=CU + 1), 3), (dict(cu=0), 1),  # 10 rows for 3 sequences
    (dict(strides=(128, -64, 128, 64)), 1), (dict(strides=(128, 64, 132, 64)), 3),
    (dict(B=0), 0), (dict(T=0), 0),
], ids=str)
def test_write_refusals(kw, status):
    assert write(**kw) == status


def test_write_refuses_bad_rows():
    assert write(k=0) == 1 and write(v=0) == 1
    assert write(k=KN + 8) == 3
    assert write(k=V) == 1 and write(v=MS) == 1  # rows inside the cache
    assert fa.fa_cache_write_raw(None, KN, VN, 128, 64, 128, 64, CU, LENS, TABLE, 9, 9, 3, 10, 1, None) == 1


def read(c={}, k=KN, v=VN, lens=LENS, table=TABLE, table_stride=9, P=9, B=3, N=50, dtype=0):
    return fa.fa_cache_read_raw(ctypes.byref(desc(**c)), k, v, lens, table, table_stride, P, B, N, dtype, None)


@pytest.mark.parametrize("kw,status", BAD_CACHES + [
    (dict(dtype=5), 2), (dict(B=-1), 1), (dict(N=-1), 1), (dict(lens=0), 1), (dict(P=0), 1), (dict(B=65536), 2),
    (dict(B=60000, N=1 << 27), 2), (dict(B=0), 0), (dict(N=0), 0),
], ids=str)
def test_read_refusals(kw, status):
    assert read(**kw) == status


def test_read_refuses_bad_outputs():
    assert read(k=0) == 1
    assert read(v=VN + 8) == 3
    assert read(k=K) == 1 and read(v=KN + 64) == 1 and read(k=TABLE) == 1


def decode(c={}, q=Q, strides=(256, 64, 64), o=O, lse=L, lens=LENS, table=TABLE, table_stride=9, P=9, pages=PAGES,
           slots=4, ws=W, ws_bytes=1 << 30, B=3, Hq=4, Nq=1, scale=0.125, causal=0, dtype=0):
    return fa.fa_decode_cache_raw(ctypes.byref(desc(**c)), q, *strides, o, lse, lens, table, table_stride, P,
                                  pages, slots, ws, ws_bytes, B, Hq, Nq, scale, causal, dtype, None)


QUERIES = [
    (dict(Nq=0), 2), (dict(Nq=17), 2), (dict(Hq=3), 1), (dict(causal=2), 1), (dict(dtype=9), 2), (dict(q=0), 1),
    (dict(q=Q + 8), 3), (dict(strides=(256, 60, 64)), 3), (dict(strides=(-256, 64, 64)), 1), (dict(lens=0), 1),
    (dict(table_stride=3), 1), (dict(B=-1), 1), (dict(Hq=-4), 1), (dict(ws=0), 1), (dict(ws=W + 4), 3),
    (dict(ws_bytes=8), 1), (dict(pages=PAGES + 2), 3), (dict(ws=K), 1), (dict(ws=Q), 1), (dict(B=0), 0), (dict(Hq=0), 0),
]


@pytest.mark.parametrize("kw,status", BAD_CACHES + QUERIES + [
    (dict(scale=float("nan")), 1), (dict(scale=-1.0), 2), (dict(slots=0), 1), (dict(o=0), 1), (dict(o=O + 8), 3),
    (dict(lse=L + 1), 3), (dict(o=V), 1), (dict(o=Q), 1), (dict(lse=O), 1), (dict(ws=O), 1), (dict(o=PAGES), 1),
], ids=str)
def test_decode_refusals(kw, status):
    assert decode(**kw) == status


def select(c={}, q=Q, strides=(256, 64, 64), lens=LENS, table=TABLE, table_stride=9, P=9, pages=PAGES, slots=4,
           first=1, last=1, ws=W, ws_bytes=1 << 30, B=3, Hq=4, Nq=1, causal=0, dtype=0):
    return fa.fa_cache_select_raw(ctypes.byref(desc(**c)), q, *strides, lens, table, table_stride, P, pages,
                                  slots, first, last, ws, ws_bytes, B, Hq, Nq, causal, dtype, None)


@pytest.mark.parametrize("kw,status", BAD_CACHES + QUERIES + [
    (dict(c=dict(k_mean=0, k_mean_scale=0)), 1), (dict(first=-1), 1), (dict(last=0), 1), (dict(slots=1), 1),
    (dict(first=2147483647, last=2147483647), 1), (dict(pages=0), 1), (dict(pages=M), 1), (dict(pages=LENS), 1),
    (dict(pages=W), 1),
], ids=str)
def test_select_refusals(kw, status):
    assert select(**kw) == status


def test_workspace_sizes():
    assert fa.fa_cache_select_workspace_size(3, 2, 4, 9) == 3 * 2 * 4 * 9 * 4
    assert fa.fa_cache_select_workspace_size(3, 2, 17, 9) == 0
    assert fa.fa_decode_cache_workspace_size(3, 4, 2, 1, 64) > 0
    assert fa.fa_decode_cache_workspace_size(3, 5, 2, 1, 64) == 0
    assert fa.fa_decode_cache_workspace_size(3, 4, 2, 17, 64) == 0
    assert fa.fa_decode_cache_workspace_size(3, 4, 2, 1, 48) == 0


def test_python_refuses_cpu_tensors_and_wrong_types():
    cache = fa.FACache.empty(4, 2, 16, 32, device="cpu")
    x = torch.zeros(3, 2, 32, dtype=torch.bfloat16)
    table, lens = torch.zeros(3, 4, dtype=torch.int32), torch.zeros(3, dtype=torch.int32)
    q = torch.zeros(3, 4, 1, 32, dtype=torch.bfloat16)
    for call in (lambda: fa.fa_cache_write(cache, x, x, table, lens), lambda: fa.fa_cache_read(cache, table, lens, 5),
                 lambda: fa.fa_decode_cache(q, cache, table, lens), lambda: fa.fa_cache_select(q, cache, table, lens, 3),
                 lambda: fa.fa_decode_cache(q, tuple(cache), table, lens),
                 lambda: fa.FACache.empty(4, 2, 16, 32, dtype=torch.float16, device="cpu")):
        with pytest.raises(fa.FAError):
            call()


def test_definition_by_hand():
    assert scale_of(448.0, 448.0) == 1.0 and scale_of(449.0, 448.0) == 2.0 and scale_of(224.0, 448.0) == 0.5
    assert scale_of(127.0, 127.0) == 1.0 and scale_of(0.0, 448.0) == 2.0 ** -60 == scale_of(1e-30, 448.0)
    x = torch.tensor([17.0, 19.0, 2.0 ** -10, 3 * 2.0 ** -10, 500.0, -math.inf], dtype=torch.float64)
    assert encode(x, "e4m3").tolist() == [16.0, 20.0, 0.0, 2.0 ** -8, 448.0, -448.0]
    assert encode(torch.tensor([0.5, 1.5, -2.5, 300.0], dtype=torch.float64), "int8").tolist() == [0.0, 2.0, -2.0, 127.0]
    assert math.isnan(encode(torch.tensor([math.nan]).double(), "e4m3")[0])
    # two tokens of one head, e4m3: the second one's page scale grows and moves the first one's codes
    ref = Ref(1, 1, 16, 32, "e4m3")
    k = torch.zeros(2, 1, 32)
    k[0, 0, 0], k[0, 0, 1], k[1, 0, 2] = 448.0, 17.0, 448.0 * 64
    ref.write(k[:1], k[:1], torch.zeros(1, 1, dtype=torch.int32), [0], [0, 1])
    assert float(ref.k_scale[0, 0]) == 1.0 and ref.k[0, 0, 0, :2].tolist() == [448.0, 16.0]
    ref.write(k[1:], k[1:], torch.zeros(1, 1, dtype=torch.int32), [1], [0, 1])
    assert float(ref.k_scale[0, 0]) == 64.0
    assert ref.k[0, 0, 0, :2].tolist() == [7.0, 0.25] and ref.k[0, 0, 1, 2] == 448.0
    # attention with one key is its value, and with two equal keys their mean
    ref.v[0, 0, 0], ref.v[0, 0, 1] = 2.0, 4.0
    ref.k[0, 0, 1] = ref.k[0, 0, 0]
    ref.v_scale[0, 0] = 0.5
    q = torch.ones(1, 1, 1, 32)
    for n, want in ((1, 1.0), (2, 1.5)):
        o, lse, a, _ = ref.attend(q, torch.zeros(1, 1, dtype=torch.int32), [n], 0.25, False)
        assert torch.allclose(o, torch.full_like(o, want))
        assert math.isclose(float(lse), 0.25 * 64 * 7.25 + math.log(n))
    # the summary of a page, and the score it gives
    ref.k[0, 0] = 0.0
    ref.k[0, 0, :, 3] = torch.arange(16.0).double()
    ref.summarise(0, 0)
    assert ref.k_mean[0, 0, 3] == 120.0 and float(ref.k_mean_scale[0, 0]) == 2.0 ** -4 * 64
