"""Rotary positions, page plans and the 4-bit cache through the CPython module and through ctypes: the same results, and
the same refusals."""
import pytest
import torch

import attention_forward_02_gb300 as fa
from attention_forward_02_gb300 import cache as module

pytestmark = pytest.mark.gpu
DEV = "cuda"


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def everything():
    """Outputs of usual calls, and what unusual ones say."""
    g = torch.Generator(device=DEV).manual_seed(1)
    rand = lambda *shape, dtype=torch.bfloat16: torch.randn(shape, generator=g, device=DEV).to(dtype)  # noqa: E731
    outs, said = [], []
    H, d, page, B, T = 2, 64, 16, 3, 40
    pool, table = fa.FAPagePool.full(12), torch.full((B, 4), -1, dtype=torch.int32, device=DEV)
    lens, new = i32([0, 0, 0]), i32([20, 1, 15])
    plan = fa.fa_cache_plan(pool, table, lens, new, page, T)
    assert type(plan) is fa.FAPlan
    kept = torch.empty(2, dtype=torch.int64, device=DEV)
    again = fa.fa_cache_plan(pool, table.clone(), plan.ends, new, page, T, counts=kept)
    outs += [*plan, *again, kept, table, pool.counts.clone()]
    rope = fa.FARope.new(32, interleaved=True)
    x = rand(T, 8 + 2 * H, d)
    q, k = fa.fa_rope(x[:, :8], x[:, 8:8 + H], rope, plan.positions)
    alone, none = fa.fa_rope(x[:, :8], None, rope, plan.positions, backward=True)
    assert none is None
    inplace = x.clone()
    given = fa.fa_rope(inplace[:, :8], inplace[:, 8:10], rope, plan.positions, q_out=inplace[:, :8], k_out=inplace[:, 8:10])
    assert given[0].data_ptr() == inplace.data_ptr()
    heads = rand(2, 3, 17, d, dtype=torch.float16)
    outs += [q, k, alone, inplace, *fa.fa_rope(heads, heads[:, :1], rope),
             fa.fa_rope(heads, None, rope, torch.arange(34, dtype=torch.int32, device=DEV).view(2, 17))[0],
             fa.fa_rope(heads, None, rope, torch.arange(17, dtype=torch.int32, device=DEV))[0]]
    c = fa.FACache4(torch.zeros(12, H, page, d // 8 * 9, dtype=torch.uint8, device=DEV))
    fa.fa_cache4_write(c, k, x[:, 8 + H:], plan.slots)
    outs += [c.data.clone(), *fa.fa_cache4_read(c, table, plan.ends, 25), *fa.fa_cache4_read(c, table, plan.ends, 25, dtype=torch.float16)]
    k16 = torch.empty(B, H, 9, d, dtype=torch.float16, device=DEV)
    got = fa.fa_cache4_read(c, table, plan.ends, 9, k=k16)
    assert got[0] is k16 and got[1].dtype is torch.float16
    outs += got
    qd = rand(B, 2, 8, d).transpose(1, 2)
    o, lse = fa.fa_decode_cache4(qd, c, table, plan.ends, causal=True, scale=0.2)
    ws = torch.empty(fa.fa_decode_cache4_workspace_size(B, 8, H, 2, d), dtype=torch.uint8, device=DEV)
    o2 = torch.empty_like(o)
    got = fa.fa_decode_cache4(qd, c, table, plan.ends, o=o2, return_lse=False, workspace=ws)
    assert got[0] is o2 and got[1] is None
    outs += [o, lse, o2]
    fa.fa_cache_trim(pool, table, plan.ends, i32([3, 0, 15]), page)
    outs += [pool.ring.clone(), pool.counts.clone()]

    odd = torch.zeros(T, 8, d + 1, device=DEV, dtype=torch.bfloat16)[:, :, 1:]
    calls = [
        lambda: fa.fa_cache_plan(pool, table, lens, new, 48, T), lambda: fa.fa_cache_plan(pool, table, lens, new, page, -1),
        lambda: fa.fa_cache_plan(pool, table, lens, new, page, 2 ** 31), lambda: fa.fa_cache_plan(pool, table, lens, new[:2], page, T),
        lambda: fa.fa_cache_plan(pool, table, lens.long(), new, page, T), lambda: fa.fa_cache_plan(pool, table, lens, lens, page, T, counts=lens),
        lambda: fa.fa_cache_plan(fa.FAPagePool(pool.ring.long(), pool.counts), table, lens, new, page, T),
        lambda: fa.fa_cache_trim(pool, table, lens, new, 8), lambda: fa.fa_cache_trim(pool, table.t(), lens, new, page),
        lambda: fa.fa_rope(x[:, :8], k[:5], rope, plan.positions), lambda: fa.fa_rope(x[:, :8], k.half(), rope, plan.positions),
        lambda: fa.fa_rope(x[:, :8].float(), None, rope), lambda: fa.fa_rope(x[0], None, rope), lambda: fa.fa_rope(odd, None, rope),
        lambda: fa.fa_rope(x[:, :8], None, rope, plan.positions[:3]), lambda: fa.fa_rope(x[:, :8], None, rope, plan.positions.long()),
        lambda: fa.fa_rope(x[:, :8], None, rope, q_out=x[:, 1:9]), lambda: fa.fa_rope(x[:, :8], None, rope, k_out=x[:, :8]),
        lambda: fa.fa_rope(x[:, :8], None, fa.FARope(rope.turns.int())), lambda: fa.fa_rope(x[:, :8], None, rope, q_out=q.half()),
        lambda: fa.fa_rope(x[:, :8], None, fa.FARope(rope.turns[:6])), lambda: fa.fa_rope(x[:, :8], None, (rope.turns, True, 1.0)),
        lambda: fa.fa_cache4_write(c, k, x[:, 8 + H:], plan.slots[:4]), lambda: fa.fa_cache4_write(c, k[:, :1], k[:, :1], plan.slots),
        lambda: fa.fa_cache4_write(c, k.float(), k.float(), plan.slots), lambda: fa.fa_cache4_write(fa.FACache4(c.data[:, :, :, :64]), k, k, plan.slots),
        lambda: fa.fa_cache4_read(c, table, plan.ends, -1), lambda: fa.fa_cache4_read(c, table, plan.ends, 2 ** 31 + 5),
        lambda: fa.fa_cache4_read(c, table, plan.ends, 5, dtype=torch.float32), lambda: fa.fa_cache4_read(c, table, plan.ends, 9, k=k16, v=k16),
        lambda: fa.fa_decode_cache4(qd[:, :5], c, table, plan.ends), lambda: fa.fa_decode_cache4(qd[:2], c, table, plan.ends),
        lambda: fa.fa_decode_cache4(qd, c, table, plan.ends, scale=-1.0), lambda: fa.fa_decode_cache4(qd, c, table, plan.ends, workspace=ws[:64]),
        lambda: fa.fa_decode_cache4(rand(B, 8, 17, d), c, table, plan.ends), lambda: fa.fa_decode_cache4(qd, c.data, table, plan.ends),
        lambda: fa.fa_decode_cache4(qd, c, table, plan.ends, o=qd),
    ]
    for f in calls:
        with pytest.raises(fa.FAError) as e:
            f()
        said.append((e.value.status, str(e.value)))
    torch.cuda.synchronize()
    return outs, said


def test_both_ways_agree(monkeypatch):
    assert module._quick(), "the CPython module is not built"
    quick, quick_said = everything()
    monkeypatch.setattr(module, "_module", False)
    monkeypatch.setattr(module, "_bound", fa.load())
    assert not module._quick()
    longer, longer_said = everything()
    assert quick_said == longer_said
    for x, y in zip(quick, longer, strict=True):
        assert x.dtype == y.dtype and x.shape == y.shape and torch.equal(x, y)


def test_outputs_of_one_allocation():
    """Contiguous, apart from one another, on 16-byte borders, and in place of their memory when written to."""
    rope, lens = fa.FARope.new(32), i32([0, 0, 0])
    x = torch.randn(5, 7, 32, device=DEV, dtype=torch.float16)
    pool, table = fa.FAPagePool.full(9), torch.zeros(3, 4, dtype=torch.int32, device=DEV)
    plan = fa.fa_cache_plan(pool, table, lens, i32([3, 1, 2]), 16, 7)
    cache = fa.FACache4(torch.zeros(9, 3, 16, 36, dtype=torch.uint8, device=DEV))
    for group in (fa.fa_rope(x, x[:, :3], rope), fa.fa_cache4_read(cache, table, plan.ends, 5), plan):
        spans = sorted((t.data_ptr(), t.data_ptr() + t.nbytes) for t in group)
        assert all(a[1] <= b[0] for a, b in zip(spans, spans[1:]))
        for t in group:
            assert t.is_contiguous() and t.data_ptr() % 16 == 0 and not t.requires_grad
            others = [u.clone() for u in group if u is not t]
            t.add_(1).view(-1)[-1:].zero_()
            assert all(torch.equal(u, v) for u, v in zip(others, [u for u in group if u is not t]))
            assert t.storage_offset() * t.element_size() + t.nbytes <= t.untyped_storage().nbytes()


def test_large_outputs_have_memory_of_their_own():
    """Either may be freed or saved without the other."""
    rope = fa.FARope.new(128)
    x = torch.randn(600, 8, 128, device=DEV, dtype=torch.float16)
    cache = fa.FACache4(torch.zeros(9, 3, 128, 144, dtype=torch.uint8, device=DEV))
    table = torch.zeros(1, 6, dtype=torch.int32, device=DEV)
    for group in (fa.fa_rope(x, x[:, :3], rope), fa.fa_cache4_read(cache, table, i32([700]), 768)):
        for t in group:
            assert t.untyped_storage().nbytes() < 2 * t.nbytes and t.storage_offset() == 0
        assert group[0].untyped_storage().data_ptr() != group[1].untyped_storage().data_ptr()


def test_streams_and_empty_calls_go_the_longer_way():
    rope = fa.FARope.new(64)
    x = torch.randn(5, 2, 64, device=DEV, dtype=torch.float16)
    want, _ = fa.fa_rope(x, None, rope)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got, _ = fa.fa_rope(x, None, rope, stream=side)
    side.synchronize()
    assert torch.equal(got, want)
    empty, _ = fa.fa_rope(x[:0], None, rope)
    assert empty.shape == (0, 2, 64)
    with pytest.raises(fa.FAError):
        fa.fa_rope(x.cpu(), None, rope)
