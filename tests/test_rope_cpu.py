"""fa_rope: what the call refuses before any CUDA call, and the frequencies of FARope.new."""
import ctypes
import itertools
import math

import pytest
import torch

import attention_forward_02_gb300 as fa
from attention_forward_02_gb300.build import build_library
from attention_forward_02_gb300.rope import _scaled
from rope_util import turn

Q, QO, K, KO, TURNS, POS = 0x10000000, 0x20000000, 0x30000000, 0x40000000, 0x50000000, 0x60000000


@pytest.fixture(scope="module", autouse=True)
def lib():
    build_library()
    return fa.load()


def call(pairs=32, interleaved=0, factor=1.0, turns=TURNS, q=Q, qo=QO, k=K, ko=KO, Hq=8, H=2, B=2, N=5, d=64,
         q_in=None, q_out=None, k_in=None, k_out=None, pos=POS, pos_stride=5, backward=0, dtype=0, no_k=False):
    rope = fa.RopeDesc(turns, pairs, interleaved, factor)
    rq = fa.RopeRows(q, qo, *(q_in or (Hq * N * d, N * d, d)), *(q_out or (Hq * N * d, N * d, d)), Hq)
    rk = fa.RopeRows(k, ko, *(k_in or (H * N * d, N * d, d)), *(k_out or (H * N * d, N * d, d)), H)
    return fa.fa_rope_raw(ctypes.byref(rope), ctypes.byref(rq), None if no_k else ctypes.byref(rk), pos, pos_stride, B, N,
                          d, backward, dtype, None)


@pytest.mark.parametrize("kwargs,status", [
    (dict(d=48), 2), (dict(dtype=2), 2), (dict(pairs=30), 2), (dict(pairs=36), 2), (dict(pairs=0), 1), (dict(pairs=-4), 1),
    (dict(factor=float("nan")), 1), (dict(factor=float("inf")), 1), (dict(interleaved=2), 1), (dict(backward=2), 1),
    (dict(B=-1), 1), (dict(N=-1), 1), (dict(Hq=-1), 1), (dict(H=-1), 1),
    (dict(Hq=65536), 2), (dict(H=2 ** 31 - 1), 2), (dict(N=2 ** 30, q_in=(64, 64, 1 << 34)), 1),
    (dict(B=2 ** 30, pos_stride=1 << 34), 1),
    (dict(turns=0), 1), (dict(q=0), 1), (dict(qo=0), 1), (dict(k=0), 1), (dict(ko=0), 1),
    (dict(q=Q + 8), 3), (dict(qo=QO + 2), 3), (dict(turns=TURNS + 4), 3), (dict(pos=POS + 2), 3),
    (dict(q_in=(8 * 5 * 64, 5 * 64, 66)), 3), (dict(k_out=(1000, 500, 68)), 3),
    (dict(q_in=(-64, 5 * 64, 64)), 1), (dict(q_in=(1 << 41, 5 * 64, 64)), 1), (dict(pos_stride=-1), 1),
    (dict(q_out=(0, 5 * 64, 64)), 1),            # two batches in one place
    (dict(q_out=(8 * 5 * 64, 64, 64)), 1),       # heads over rows
    (dict(qo=Q + 64), 1),                        # output over its input, elsewhere
    (dict(qo=Q, q_out=(8 * 5 * 64, 64, 8 * 64)), 1),  # in place, other strides
    (dict(ko=QO + 512), 1), (dict(ko=Q), 1), (dict(qo=K), 1),
    (dict(qo=TURNS), 1), (dict(ko=POS), 1),
    (dict(N=0), 0), (dict(B=0), 0), (dict(Hq=0, H=0), 0), (dict(Hq=0, no_k=True), 0), (dict(N=0, q=0, turns=0), 0),
], ids=str)
def test_refusals(kwargs, status):
    assert call(**kwargs) == status


def test_null_structs():
    rope = fa.RopeDesc(TURNS, 32, 0, 1.0)
    rows = fa.RopeRows(Q, QO, 640, 64, 64, 640, 64, 64, 1)
    assert fa.fa_rope_raw(None, ctypes.byref(rows), None, POS, 0, 1, 1, 64, 0, 0, None) == 1
    assert fa.fa_rope_raw(ctypes.byref(rope), None, None, POS, 0, 1, 1, 64, 0, 0, None) == 1


def test_rows_side_by_side_reach_the_device():
    """Heads of one buffer side by side do not overlap: without a GPU the call gets as far as CUDA (status 4)."""
    if torch.cuda.is_available():
        pytest.skip("fake addresses would reach the GPU")
    row = 12 * 64
    s = (5 * row, 64, row)
    args = dict(q=Q, qo=Q, k=Q + 8 * 128, ko=Q + 8 * 128, q_in=s, q_out=s, k_in=s, k_out=s)
    assert call(**args) == 4
    assert call(**dict(args, k=Q + 7 * 128, ko=Q + 7 * 128)) == 1        # one head of both
    assert call(**dict(args, k=Q + 11 * 128, ko=Q + 11 * 128)) == 1      # runs into the next row
    assert call(**dict(args, k_in=(5 * row, 64, row + 64), k_out=(5 * row, 64, row + 64))) == 1
    assert call(**dict(args, q_in=(4 * row, 64, row), q_out=(4 * row, 64, row), k_in=(4 * row, 64, row),
                       k_out=(4 * row, 64, row))) == 1                   # batches into one another


def test_python_refusals():
    rope = fa.FARope.new(64, device="cpu")
    x = torch.zeros(4, 2, 64, dtype=torch.float16)
    with pytest.raises(fa.FAError, match="CUDA tensor"):
        fa.fa_rope(x, None, rope)
    for args in (dict(rot=12), dict(rot=0), dict(rot=8.0), dict(rot=8, scaling="other"), dict(rot=8, base=-1.0),
                 dict(rot=8, scaling="yarn"), dict(rot=8, scaling="linear", factor=0.0), dict(rot=8, radians=[1.0]),
                 dict(rot=8, radians=[1.0, float("nan"), 1.0, 1.0]), dict(rot=8, scaling="bands", trained=10, fast=1.0),
                 dict(rot=8, base=1.0, scaling="yarn", trained=100), dict(rot=64, base=1e300, scaling="base", factor=1e300),
                 dict(rot=8, scaling="yarn", trained=100, fast=float("inf")), dict(rot=8, base=float("nan"))):
        with pytest.raises(fa.FAError):
            fa.FARope.new(device="cpu", **args)


def test_turns_are_the_radians():
    rope = fa.FARope.new(128, device="cpu")
    for i, t in enumerate(rope.turns.tolist()):
        w = 10000.0 ** (-2.0 * i / 128)
        assert abs((t % 2 ** 64) / 2.0 ** 64 - w / (2 * math.pi)) <= 2.0 ** -52
    # whole turns mean nothing, and negative angles turn the other way
    a = fa.FARope.new(8, radians=[0.25, -0.25, 0.25 + 2 * math.pi, 0.0], device="cpu").turns.tolist()
    assert abs(a[0] + a[1]) <= 1 and abs(a[0] - a[2]) <= 2 ** 14 and a[3] == 0


def test_scalings():
    rot, plain = 64, [10000.0 ** (-2.0 * i / 64) for i in range(32)]
    assert _scaled(rot, 10000.0, None, 8.0, None, 32.0, 1.0) == (plain, 1.0)
    w, f = _scaled(rot, 10000.0, "linear", 8.0, None, 32.0, 1.0)
    assert f == 1.0 and all(math.isclose(a * 8, b) for a, b in zip(w, plain))
    w, f = _scaled(rot, 10000.0, "base", 8.0, None, 32.0, 1.0)
    assert f == 1.0 and w[0] == 1.0 and math.isclose(w[-1] * 8, plain[-1])
    for kind in ("yarn", "bands"):
        w, f = _scaled(rot, 10000.0, kind, 8.0, 4096, 32.0, 1.0)
        assert math.isclose(f, 0.1 * math.log(8.0) + 1.0 if kind == "yarn" else 1.0)
        for a, b in zip(w, plain):
            turns = 4096 * b / (2 * math.pi)
            assert b / 8 * (1 - 1e-12) <= a <= b * (1 + 1e-12)
            if turns > 50:
                assert math.isclose(a, b)
            if turns < 0.7:
                assert math.isclose(a * 8, b)
        assert all(x > y for x, y in zip(w, w[1:]))


@pytest.mark.parametrize("interleaved", [False, True])
def test_definition(interleaved):
    """The reference itself: one pair by hand, lengths kept, and the gradient against central differences."""
    turns = [2 ** 62, 2 ** 60, 2 ** 50, -2 ** 61]  # a quarter turn a position, ...
    pos = torch.tensor([[1, 3]])
    x = torch.randn(1, 1, 2, 16, generator=torch.Generator().manual_seed(0), dtype=torch.float64)
    y, _ = turn(x, turns, interleaved, 1.0, pos)
    a, b = (0, 1) if interleaved else (0, 4)
    assert torch.allclose(y[0, 0, 0, [a, b]], torch.stack((-x[0, 0, 0, b], x[0, 0, 0, a])), atol=1e-12)
    assert torch.allclose(y[0, 0, 1, [a, b]], torch.stack((x[0, 0, 1, b], -x[0, 0, 1, a])), atol=1e-12)
    assert torch.allclose(y.norm(), x.norm()) and torch.equal(y[..., 8:], x[..., 8:])
    g = torch.randn_like(x)
    back, _ = turn(g, turns, interleaved, 1.0, pos, backward=True)
    for at in itertools.product(range(2), range(16)):
        h = torch.zeros_like(x)
        h[0, 0][at] = 1e-3
        up, down = (turn(x + s * h, turns, interleaved, 1.0, pos)[0] for s in (1, -1))
        assert abs(float(((up - down) * g).sum()) / 2e-3 - float(back[0, 0][at])) < 1e-9
