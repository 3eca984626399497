"""fa_rope on the GPU against the definition in 64 bits, element by element."""
import pytest
import torch

import attention_forward_02_gb300 as fa
from rope_util import DTYPES, bound, turn

pytestmark = pytest.mark.gpu
DEV = "cuda"


def normal(shape, dtype, seed):
    return torch.randn(shape, generator=torch.Generator().manual_seed(seed)).to(DTYPES[dtype])


def numbers(rope):
    return [int(x) for x in rope.turns.cpu()]


def check(got, x, rope, positions, backward=False):
    """got, x [B, H, N, d]; positions [B, N] on the CPU."""
    y, mag = turn(x.cpu(), numbers(rope), rope.interleaved, rope.factor, positions, backward)
    over = (got.cpu().double() - y).abs() - bound(y, mag, got.dtype)
    assert over.max() <= 0, "off by more than the bound: %g" % over.max()


@pytest.mark.parametrize("d,rot", [(32, 32), (32, 8), (64, 64), (64, 16), (96, 96), (96, 24), (96, 48), (128, 128),
                                   (128, 64), (128, 120), (128, 8)])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("backward", [False, True])
def test_tokens(d, rot, interleaved, dtype, backward):
    """Packed tokens of a fused projection, far and near positions, padding."""
    T, Hq, H = 13, 6, 2
    rope = fa.FARope.new(rot, interleaved=interleaved, scaling="yarn", factor=4.0, trained=4096)
    x = normal((T, Hq + 2 * H, d), dtype, d + rot).to(DEV)
    q, k = x[:, :Hq], x[:, Hq:Hq + H]
    before = x.clone()
    pos = torch.tensor([0, 1, 2, 131071, 5, -1, 2 ** 31 - 1, 1000003, -7, 4096, 77, 8, 9], dtype=torch.int32)
    yq, yk = fa.fa_rope(q, k, rope, pos.to(DEV), backward=backward)
    for y, z in ((yq, q), (yk, k)):
        check(y.transpose(0, 1)[None], z.transpose(0, 1)[None], rope, pos[None], backward)
        assert torch.equal(y[pos.to(DEV) < 0], z[pos.to(DEV) < 0])
        assert torch.equal(y[..., rot:], z[..., rot:])
    assert torch.equal(x, before)


@pytest.mark.parametrize("d,rot", [(32, 32), (32, 8), (64, 64), (64, 16), (96, 96), (96, 24), (128, 128), (128, 56)])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("T,Hq,H", [(1, 32, 8), (3, 29, 5), (9, 64, 8), (40, 24, 3), (200, 16, 1)])
@pytest.mark.parametrize("backward", [False, True])
def test_few_tokens_of_many_heads(d, rot, interleaved, T, Hq, H, backward):
    rope = fa.FARope.new(rot, interleaved=interleaved)
    x = normal((T, Hq + H, d), "bf16", d + rot).to(DEV)
    pos = torch.tensor([[131071, -1, 2 ** 31 - 1, 0, 5][t % 5] if t % 3 else t for t in range(T)], dtype=torch.int32)
    y = torch.full_like(x, 7.0)
    fa.fa_rope(x[:, :Hq], x[:, Hq:], rope, pos.to(DEV), q_out=y[:, :Hq], k_out=y[:, Hq:], backward=backward)
    check(y.transpose(0, 1)[None], x.transpose(0, 1)[None], rope, pos[None], backward)
    assert torch.equal(y[pos.to(DEV) < 0], x[pos.to(DEV) < 0]) and torch.equal(y[..., rot:], x[..., rot:])


@pytest.mark.parametrize("B,Hq,H,N,d", [(1, 1, 1, 1, 128), (2, 3, 3, 65, 64), (3, 8, 1, 7, 32), (1, 40, 8, 1, 128),
                                        (2, 5, 0, 33, 96), (1, 0, 4, 9, 64), (4, 128, 2, 1, 128), (1, 2, 2, 1500, 128)])
@pytest.mark.parametrize("kind", ["none", "row", "each"])
def test_heads(B, Hq, H, N, d, kind):
    """[B, H, N, d] as fa_fwd takes it, positions counted, shared by the batch, or each its own."""
    rope = fa.FARope.new(d // 2 if d != 96 else 96, interleaved=bool(N % 2))
    q, k = normal((B, Hq, N, d), "fp16", 1).to(DEV), normal((B, H, N, d), "fp16", 2).to(DEV)
    pos = torch.arange(N)[None].expand(B, N)
    given = None
    if kind == "row":
        pos = (torch.arange(N) * 37 % 1001)[None].expand(B, N)
        given = pos[0].int().to(DEV)
    elif kind == "each":
        wide = torch.randint(0, 50000, (B, N + 3), generator=torch.Generator().manual_seed(3))
        given = wide.int().to(DEV)[:, :N]
        pos = wide[:, :N]
    yq, yk = fa.fa_rope(q, k, rope, given)
    if Hq:
        check(yq, q, rope, pos)
    if H:
        check(yk, k, rope, pos)
    alone, none = fa.fa_rope(q, None, rope, given)
    assert none is None and torch.equal(alone, yq)


def test_in_place_side_by_side():
    """Query and key rows of one buffer, turned where they lie; the value rows stay."""
    rope = fa.FARope.new(128)
    x = normal((300, 12, 128), "bf16", 5).to(DEV)
    before = x.clone()
    pos = torch.arange(300, dtype=torch.int32, device=DEV) * 11
    wq, wk = fa.fa_rope(before[:, :8], before[:, 8:10], rope, pos)
    yq, yk = fa.fa_rope(x[:, :8], x[:, 8:10], rope, pos, q_out=x[:, :8], k_out=x[:, 8:10])
    assert yq.data_ptr() == x.data_ptr()
    assert torch.equal(x[:, :8], wq) and torch.equal(x[:, 8:10], wk) and torch.equal(x[:, 10:], before[:, 10:])
    # [B, H, N, d] views of a [B, N, heads, d] buffer
    z = normal((2, 50, 12, 64), "fp16", 6).to(DEV)
    was = z.clone()
    rope = fa.FARope.new(64, interleaved=True)
    q, k = z[:, :, :8].transpose(1, 2), z[:, :, 8:10].transpose(1, 2)
    wq, wk = fa.fa_rope(was[:, :, :8].transpose(1, 2), was[:, :, 8:10].transpose(1, 2), rope)
    fa.fa_rope(q, k, rope, q_out=q, k_out=k)
    assert torch.equal(q, wq) and torch.equal(k, wk) and torch.equal(z[:, :, 10:], was[:, :, 10:])


def test_broadcast_input():
    """One key head read for four (stride 0), each written."""
    rope = fa.FARope.new(64)
    k = normal((20, 1, 64), "bf16", 8).to(DEV)
    pos = torch.arange(20, dtype=torch.int32, device=DEV)
    y, _ = fa.fa_rope(k.expand(20, 4, 64), None, rope, pos)
    one, _ = fa.fa_rope(k, None, rope, pos)
    assert torch.equal(y, one.expand(20, 4, 64))


@pytest.mark.parametrize("interleaved", [False, True])
def test_gradient_by_differences(interleaved):
    """The map is linear: its columns are the outputs of unit steps, and the gradient of each output is a row."""
    d, rot = 32, 24
    rope = fa.FARope.new(rot, interleaved=interleaved, scaling="yarn", factor=8.0, trained=1024)
    pos = torch.full((d,), 12345, dtype=torch.int32, device=DEV)
    unit = torch.eye(d, dtype=torch.float16, device=DEV)[:, None]  # step c is token c
    y, _ = fa.fa_rope(unit, None, rope, pos)
    g, _ = fa.fa_rope(unit, None, rope, pos, backward=True)
    # y[c, j]: output j by input c; g[j, c]: the gradient of output j by input c
    assert torch.equal(y[:, 0], g[:, 0].t())
    # and with values: <y(x + h) - y(x), g> = <h, backward(g)>, all in 64 bits from one rounding each
    x, h, w = (normal((7, 3, d), "fp16", s) for s in (1, 2, 3))
    p = torch.arange(7, dtype=torch.int32) * 999
    yx, _ = turn((x.double() + h.double()).transpose(0, 1)[None], numbers(rope), interleaved, rope.factor, p[None])
    y0, _ = turn(x.transpose(0, 1)[None], numbers(rope), interleaved, rope.factor, p[None])
    back, _ = fa.fa_rope(w.to(DEV), None, rope, p.to(DEV), backward=True)
    left = ((yx - y0)[0].transpose(0, 1) * w.double()).sum()
    right = (h.double() * back.cpu().double()).sum()
    assert abs(left - right) <= 2.0 ** -11 * (h.double().abs() * back.cpu().double().abs()).sum() + 1e-4


def test_infinities_and_nan_stay_in_their_pair():
    rope = fa.FARope.new(64)
    x = normal((2, 1, 64), "fp16", 9)
    x[:, 0, 3], x[:, 0, 40] = float("inf"), float("nan")
    y, _ = fa.fa_rope(x.to(DEV), None, rope, torch.tensor([-1, 5], dtype=torch.int32, device=DEV))
    y = y.cpu()
    assert torch.equal(y[0].view(torch.int16), x[0].view(torch.int16))
    bad = ~torch.isfinite(y[1, 0])
    assert set(torch.nonzero(bad)[:, 0].tolist()) == {3, 35, 8, 40}


@pytest.mark.parametrize("T,heads", [(1, 1), (3, 41), (5000, 3), (40000, 1)])
def test_sizes(T, heads):
    """From fewer rows than a block to heads that each thread goes through alone; the same rows at any size."""
    rope = fa.FARope.new(128)
    x = normal((T, heads, 128), "bf16", T).to(DEV)
    pos = (torch.arange(T) * 7).int().to(DEV)
    y, _ = fa.fa_rope(x, None, rope, pos)
    for at in {0, T // 2, T - 1}:
        one, _ = fa.fa_rope(x[at:at + 1].contiguous(), None, rope, pos[at:at + 1].clone())
        assert torch.equal(y[at:at + 1], one)
    rows = sorted({0, 1 % T, T // 3, T - 1})
    check(y[rows].transpose(0, 1)[None], x[rows].transpose(0, 1)[None], rope, pos[rows].cpu()[None])


def test_graph_stream_and_wide_strides():
    rope = fa.FARope.new(64, interleaved=True)
    x = normal((9, 16, 128), "bf16", 4).to(DEV)[:, ::2, 64:]  # every other head, half of each
    pos = torch.arange(9, dtype=torch.int32, device=DEV)
    want, _ = fa.fa_rope(x, None, rope, pos)
    out = torch.zeros(9, 8, 64, dtype=torch.bfloat16, device=DEV)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    fa.fa_rope(x, None, rope, pos, q_out=out, stream=side)
    side.synchronize()
    assert torch.equal(out, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        fa.fa_rope(x, None, rope, pos, q_out=out)
    pos += 100
    graph.replay()
    again, _ = fa.fa_rope(x, None, rope, pos)
    torch.cuda.synchronize()
    assert torch.equal(out, again) and not torch.equal(out, want)


def test_before_attention():
    """Training with turned rows: o, dq and dk of rope - attention - rope's gradient against the same in 64 bits.

    Turned rows round to fp16, 2^-11 of each entry (fp32 errors are far below): a score moves by ds <= 2^-10 |q| |k|
    scale, a weight P by 2 ds P, and P rounds to fp16 for its product (2^-11).  With e = 2 ds + 2^-10:
    |o| moves by e sum P |v|, dS = P (dP - D) by E = 2 e P (|dP| + sum P |dP|) (dP has no error of its own, D
    comes from o), dQ = scale dS K by scale (E + 2^-9 |dS|) |K| with the roundings of dS and K, dK likewise.
    The gradient of the turn adds a pair's bounds; each of the three results rounds once."""
    B, H, N, d = 1, 2, 130, 64
    q, k, v, do = (normal((B, H, N, d), "fp16", s) for s in (1, 2, 3, 4))
    rope = fa.FARope.new(d)
    pos = torch.arange(5000, 5000 + N, dtype=torch.int32)
    rq, rk = fa.fa_rope(q.to(DEV), k.to(DEV), rope, pos.to(DEV))
    o, lse = fa.fa_fwd(rq, rk, v.to(DEV), causal=True)
    dq, dk, _ = fa.fa_bwd(rq, rk, v.to(DEV), o, lse, do.to(DEV), causal=True)
    dq, dk = fa.fa_rope(dq, dk, rope, pos.to(DEV), backward=True)

    tq, tk = (turn(x, numbers(rope), False, 1.0, pos[None])[0] for x in (q, k))
    v, do, scale = v.double(), do.double(), d ** -0.5
    live = torch.ones(N, N, dtype=torch.bool).tril()
    P = torch.softmax(((tq @ tk.transpose(-1, -2)) * scale).masked_fill(~live, float("-inf")), -1)
    dP = do @ v.transpose(-1, -2)
    dS = P * (dP - (P * dP).sum(-1, keepdim=True))
    ds = 2.0 ** -10 * float(tq.norm(dim=-1).max() * tk.norm(dim=-1).max()) * scale
    e = 2 * ds + 2.0 ** -10
    E = 2 * e * P * (dP.abs() + (P * dP.abs()).sum(-1, keepdim=True)) + 2.0 ** -9 * dS.abs()
    want_q, want_k = scale * (dS @ tk), scale * (dS.transpose(-1, -2) @ tq)
    off_q, off_k = scale * (E @ tk.abs()), scale * (E.transpose(-1, -2) @ tq.abs())
    assert ((o.cpu().double() - P @ v).abs() <= (e + 2.0 ** -10) * (P @ v.abs()) + 1e-6).all()
    for got, want, off in ((dq, want_q, off_q), (dk, want_k, off_k)):
        want, _ = turn(want, numbers(rope), False, 1.0, pos[None], backward=True)
        off = off + 2.0 ** -11 * (want.abs() + off)
        both = off[..., :d // 2] + off[..., d // 2:]
        assert ((got.cpu().double() - want).abs() <= torch.cat((both, both), -1) + 2.0 ** -10 * want.abs() + 1e-6).all()
