"""The 4-bit cache: what its calls refuse before any CUDA call, and the definition that the GPU tests use."""
import ctypes
import math

import pytest
import torch

import attention_forward_02_gb300 as fa
from attention_forward_02_gb300.build import build_library
from cache4_util import E2M1, SCALES, Ref, attend_bounds, encode, value

DATA, K, V, SLOTS, LENS, TABLE, Q, O, LSE, WS = (0x1000000000 * (i + 1) for i in range(10))


@pytest.fixture(scope="module", autouse=True)
def lib():
    build_library()
    return fa.load()


def desc(data=DATA, num_pages=10, heads=2, page=16, d=64):
    return fa.Cache4Desc(data, num_pages, heads, page, d)


def split(kw):
    return {k: kw.pop(k) for k in list(kw) if k in ("data", "num_pages", "heads", "page", "d")}


def write(k=K, v=V, ks=(128, 64), vs=(128, 64), slots=SLOTS, T=5, dtype=0, **kw):
    return fa.fa_cache4_write_raw(ctypes.byref(desc(**split(kw))), k, v, *ks, *vs, slots, T, dtype, None)


def read(k=K, v=V, lens=LENS, table=TABLE, stride=4, P=4, B=2, N=20, dtype=0, **kw):
    return fa.fa_cache4_read_raw(ctypes.byref(desc(**split(kw))), k, v, lens, table, stride, P, B, N, dtype, None)


def decode(q=Q, qs=(512, 64, 64), o=O, lse=LSE, lens=LENS, table=TABLE, stride=4, P=4, ws=WS, ws_bytes=1 << 40, B=2, Hq=8,
           Nq=1, scale=0.1, causal=0, dtype=0, **kw):
    return fa.fa_decode_cache4_raw(ctypes.byref(desc(**split(kw))), q, *qs, o, lse, lens, table, stride, P, ws, ws_bytes, B,
                                   Hq, Nq, scale, causal, dtype, None)


CACHE = [(dict(data=0), 1), (dict(data=DATA + 8), 3), (dict(num_pages=0), 1), (dict(heads=0), 1), (dict(page=48), 2),
         (dict(page=8), 2), (dict(d=48), 2), (dict(d=256), 2), (dict(heads=40000), 2), (dict(num_pages=1 << 27), 2),
         (dict(num_pages=1 << 24, heads=1 << 8), 2), (dict(dtype=2), 2)]


@pytest.mark.parametrize("kwargs,status", CACHE + [
    (dict(T=-1), 1), (dict(k=0), 1), (dict(v=0), 1), (dict(slots=0), 1), (dict(k=K + 8), 3), (dict(v=V + 2), 3),
    (dict(slots=SLOTS + 2), 3), (dict(ks=(-128, 64)), 1), (dict(vs=(128, -64)), 1), (dict(ks=(132, 64)), 3),
    (dict(vs=(128, 66)), 3), (dict(k=DATA), 1), (dict(v=DATA + 256), 1), (dict(slots=DATA + 64), 1),
    (dict(T=0), 0), (dict(T=0, k=0, slots=0), 0)], ids=str)
def test_write_refusals(kwargs, status):
    assert write(**kwargs) == status


BATCH = [(dict(lens=0), 1), (dict(table=0), 1), (dict(stride=3), 1), (dict(P=0), 1), (dict(B=-1), 1), (dict(B=65536), 2),
         (dict(P=1 << 28, stride=1 << 28), 2), (dict(lens=LENS + 2), 3), (dict(table=TABLE + 2), 3)]


@pytest.mark.parametrize("kwargs,status", CACHE + BATCH + [
    (dict(N=-1), 1), (dict(k=0), 1), (dict(v=0), 1), (dict(k=K + 8), 3), (dict(v=V + 4), 3), (dict(v=K + 1024), 1),
    (dict(k=DATA), 1), (dict(v=LENS), 1), (dict(k=TABLE), 1), (dict(N=0), 0), (dict(B=0, k=0), 0),
    (dict(B=60000, N=2 ** 30), 2)], ids=str)
def test_read_refusals(kwargs, status):
    assert read(**kwargs) == status


@pytest.mark.parametrize("kwargs,status", CACHE + BATCH + [
    (dict(Hq=-8), 1), (dict(Hq=7), 1), (dict(Nq=0), 2), (dict(Nq=17), 2), (dict(scale=-0.1), 2), (dict(scale=math.nan), 1),
    (dict(scale=math.inf), 1), (dict(causal=2), 1), (dict(q=0), 1), (dict(o=0), 1), (dict(ws=0), 1), (dict(ws_bytes=100), 1),
    (dict(q=Q + 8), 3), (dict(o=O + 4), 3), (dict(ws=WS + 8), 3), (dict(lse=LSE + 2), 3), (dict(qs=(512, 64, 66), Nq=2), 3),
    (dict(qs=(-512, 64, 64)), 1), (dict(o=Q), 1), (dict(o=DATA), 1), (dict(lse=O + 64), 1), (dict(lse=LENS), 1),
    (dict(ws=DATA - 4096), 1), (dict(ws=O - 1024), 1), (dict(o=TABLE), 1),
    (dict(B=0), 0), (dict(Hq=0), 0), (dict(B=0, q=0, o=0), 0)], ids=str)
def test_decode_refusals(kwargs, status):
    assert decode(**kwargs) == status


def test_workspace_size():
    assert fa.fa_decode_cache4_workspace_size(2, 8, 2, 1, 64) > 0
    for bad in ((-1, 8, 2, 1, 64), (2, 7, 2, 1, 64), (2, 8, 0, 1, 64), (2, 8, 2, 17, 64), (2, 8, 2, 1, 48)):
        assert fa.fa_decode_cache4_workspace_size(*bad) == 0


def test_python_refusals():
    cache = fa.FACache4.empty(4, 2, 16, 64, device="cpu")
    assert cache.data.shape == (4, 2, 16, 72)
    x, n, t = torch.zeros(3, 2, 64, dtype=torch.float16), torch.zeros(3, dtype=torch.int32), torch.zeros(3, 4, dtype=torch.int32)
    for f in (lambda: fa.fa_cache4_write(cache, x, x, n), lambda: fa.fa_cache4_read(cache, t, n, 4),
              lambda: fa.fa_decode_cache4(x[None].expand(3, 3, 2, 64), cache, t, n), lambda: fa.fa_cache4_write(cache.data, x, x, n)):
        with pytest.raises(fa.FAError) as e:
            f()
        assert e.value.status == 1
    with pytest.raises(fa.FAError):
        fa.FACache4.empty(4, 2, 16, 48, device="cpu")


def test_parts():
    ref = Ref(3, 2, 32, 96)
    k, ks, v, vs = fa.FACache4(ref.bytes()).parts()
    assert torch.equal(k, (ref.k[..., 0::2] | ref.k[..., 1::2] << 4).to(torch.uint8))
    assert torch.equal(v, (ref.v[..., 0::2] | ref.v[..., 1::2] << 4).to(torch.uint8))
    assert torch.equal(ks, ref.k_scale.to(torch.uint8)) and torch.equal(vs, ref.v_scale.to(torch.uint8))


def test_definition():
    """Scale bytes are an fp16's bits 14 .. 7; values are exact in both 16-bit types; blocks by hand."""
    half = (torch.arange(0xE3, dtype=torch.int16) << 7).view(torch.float16).double()
    assert torch.equal(half, SCALES) and float(SCALES[-1]) == 10240.0
    every = (E2M1[:, None] * SCALES).flatten()
    for t in (torch.float16, torch.bfloat16):
        assert torch.equal(every.to(t).double(), every)
    x = torch.zeros(4, 16, dtype=torch.float16)
    x[0, :9] = torch.tensor([6.0, 0.25, 0.75, -1.25, 1.75, 2.5, -3.5, 5.0, 0.26])   # scale 1: ties to even numbers
    x[1, 0] = 6.25                   # 1.0417: nearest 1.0, and 6.25 saturates
    x[2, :3] = torch.tensor([float("inf"), float("nan"), 3.0])                       # scale 0.5, infinity the largest
    x[3, :2] = torch.tensor([-0.0, 2.0 ** -24])                                      # scale 0: all 0
    code, scale = encode(x)
    assert scale[:, 0].tolist() == [0x78, 0x78, 0x70, 0]
    assert code[0, :9].tolist() == [7, 0, 2, 8 + 2, 4, 4, 8 + 6, 6, 1]
    assert code[1, 0] == 7 and code[2, :3].tolist() == [7, 0, 7] and (code[3] == 0).all()
    assert value(code, scale)[0, :3].tolist() == [6.0, 0.0, 1.0]
    # a scale halfway between two: amax 6 * 1.0625 goes to the even 1.0, 6 * 1.1875 to the even 1.25
    y = torch.zeros(2, 16, dtype=torch.float16)
    y[0, 0], y[1, 0] = 6.375, 7.125
    assert encode(y)[1][:, 0].tolist() == [0x78, 0x7A]
    # bf16 beyond what fp16 holds saturates
    z = torch.full((1, 16), 1e30, dtype=torch.bfloat16)
    assert value(*encode(z))[0, 0] == 61440.0
    # a value is off by one scale at most, which is 3 / 16 of the largest of its block
    x = torch.randn(1000, 16, generator=torch.Generator().manual_seed(0)).half()
    assert ((value(*encode(x)) - x.double()).abs() <= x.double().abs().amax(-1, keepdim=True) * 0.1876).all()


def test_bounds_see_a_wrong_tile():
    """One 16-key tile of V taken from another place is beyond the bounds, and so is a wrong scale byte of K."""
    lens, d = [1000], 64
    table = torch.randperm(63, generator=torch.Generator().manual_seed(1)).int()[None]
    ref = Ref(63, 1, 16, d, seed=1)
    q = torch.randn(1, 2, 1, d, generator=torch.Generator().manual_seed(2)).to(torch.bfloat16)
    o, lse, bo, bl = attend_bounds(ref, q, table, lens, d ** -0.5, False)
    p = int(table[0, 20])
    was = ref.v[p].clone()
    ref.v[p] = ref.v[int(table[0, 21])]
    wrong = attend_bounds(ref, q, table, lens, d ** -0.5, False)
    assert ((wrong[0] - o).abs() > bo).any()
    ref.v[p] = was
    # a scale byte, twice as large, of the key with the most weight, where it adds most to its score
    k, _, _ = ref.rows(table[0], 1000)
    terms = k[0] * q[0, 0, 0].double()
    key = int(terms.sum(-1).argmax())
    block = int(terms[key].unflatten(-1, (-1, 16)).sum(-1).abs().argmax())
    ref.k_scale[int(table[0, key // 16]), 0, key % 16, block] += 8
    wrong = attend_bounds(ref, q, table, lens, d ** -0.5, False)
    assert ((wrong[1] - lse).abs() > bl).any()
