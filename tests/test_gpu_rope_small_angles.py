"""Angles near zero keep their bits: slow pairs near position 0, whose sine is all that the second channel gets.  And any
angle against 64-bit ones."""
import math

import pytest
import torch

import attention_forward_02_gb300 as fa
from rope_util import DTYPES, bound, turn

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("rows,heads", [(9, 1), (9, 40), (5000, 1)])  # a thread's and a block's sines
@pytest.mark.parametrize("interleaved", [False, True])
def test_slow_pairs(dtype, rows, heads, interleaved):
    """With channels (1, 0) a pair becomes (cos t, sin t).  The angle t, between -pi and pi, is rounded to fp32 twice, which
    moves sine and cosine by 2^-23 |t| at most (near 0, where |t| is the sine, by 2^-23 of it; near a half turn by as much of
    the angle, whatever the sine is); sincospif is good to 2 ulp of them (2^-22), the products and the sum with 0 add nothing
    but the factor's rounding (2^-24).  Then one rounding to the type."""
    w = [s * b for b in (1e-4, 1e-6, 1e-9, 3.7e-10, 1e-10, 1e-13, 1.0, math.pi) for s in (1, -1)]
    rope = fa.FARope.new(32, radians=w, interleaved=interleaved, device=DEV)
    x = torch.zeros(rows, heads, 32, dtype=DTYPES[dtype])
    x[..., slice(0, 32, 2) if interleaved else slice(0, 16)] = 1.0
    pos = torch.arange(rows, dtype=torch.int32)
    got, _ = fa.fa_rope(x.to(DEV), None, rope, pos.to(DEV))
    some = sorted({1, 2, 3, 7, 8, rows // 2, rows - 1})
    # angles in 64 bits, from whole numbers (rope_util.turn holds them in 32)
    got = got.cpu()[some].double()
    turned = [[((int(t) * p + 2 ** 63) % 2 ** 64 - 2 ** 63) / 2.0 ** 63 * math.pi for t in rope.turns.cpu()] for p in some]
    angle = torch.tensor(turned, dtype=torch.float64)
    both = torch.stack((torch.cos(angle), torch.sin(angle)), -1 if interleaved else 1)
    want = both.flatten(1)
    angle = torch.stack((angle.abs(), angle.abs()), -1 if interleaved else 1).flatten(1)
    off = 2.0 ** -23 * angle + 2.0 ** -21 * want.abs()
    fi = torch.finfo(DTYPES[dtype])
    bound = fi.eps / 2 * (want.abs() + off) + off + fi.tiny * fi.eps / 2
    for h in {0, heads - 1}:
        assert ((got[:, h] - want).abs() - bound).max() <= 0


@pytest.fixture
def wide():
    """rope_util.turn makes its angles in torch's default type."""
    torch.set_default_dtype(torch.float64)
    yield
    torch.set_default_dtype(torch.float32)


@pytest.mark.parametrize("d,rot,interleaved", [(128, 128, False), (64, 64, True), (96, 48, False), (32, 8, True)])
@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("T,heads", [(40, 3), (40, 40)])
def test_against_angles_in_64_bits(wide, d, rot, interleaved, dtype, T, heads):
    """rope_util.bound holds for an angle rounded twice, by 2^-24 of a half turn: with c and s its cosine and sine an output
    a c - b s is off by |a| (1.9e-7 |s| + 3.0e-7 |c|) + |b| (1.9e-7 |c| + 3.0e-7 |s|) at most (the angle; 2 ulp of sincospif,
    the factor and two roundings of a product and the sum), which is below 3.6e-7 < 2^-21 of |a| + |b|."""
    rope = fa.FARope.new(rot, base=500000.0, interleaved=interleaved, scaling="yarn", factor=4.0, trained=8192)
    x = torch.randn(T, heads, d, generator=torch.Generator().manual_seed(d)).to(DTYPES[dtype])
    pos = torch.tensor([(0, 1, 2, 3, 131071, 2 ** 31 - 1, 4095, 12345)[t % 8] + t // 8 * (t % 8 < 4) for t in range(T)])
    got, _ = fa.fa_rope(x.to(DEV), None, rope, pos.int().to(DEV))
    y, mag = turn(x.transpose(0, 1)[None], [int(t) for t in rope.turns.cpu()], interleaved, rope.factor, pos[None])
    over = (got.cpu().double().transpose(0, 1)[None] - y).abs() - bound(y, mag, DTYPES[dtype])
    assert over.max() <= 0
