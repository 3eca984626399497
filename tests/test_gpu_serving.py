"""A run of the operators as a serving loop uses them: pages planned, rows turned, written in 4 bits and attended to,
rejected tokens given back; and in the middle a prefix read back for a prompt's attention."""
import random

import pytest
import torch

import attention_forward_02_gb300 as fa
import pages_util
from cache4_util import Ref, attend_bounds, within
from rope_util import bound, turn

pytestmark = pytest.mark.gpu
DEV = "cuda"
H, G, D, PAGE = 2, 4, 64, 16


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


class Server:
    """The same loop in 64 bits and whole numbers on the CPU beside the calls."""

    def __init__(self, B, num_pages, wide):
        self.rope = fa.FARope.new(D, scaling="bands", factor=4.0, trained=64, fast=4.0)
        self.pool, self.cache = fa.FAPagePool.full(num_pages), fa.FACache4.empty(num_pages, H, PAGE, D)
        self.cache.data.fill_(255)  # scale bytes that are none wherever nothing was written
        self.table, self.lens = torch.full((B, wide), -1, dtype=torch.int32, device=DEV), i32([0] * B)
        self.ref = Ref(num_pages, H, PAGE, D)
        self.state = (list(range(num_pages)), [0, num_pages], [[-1] * wide for _ in range(B)], [0] * B)

    def step(self, new, pad, seed):
        g = torch.Generator().manual_seed(seed)
        T = sum(new) + pad
        qkv = torch.randn(T, G * H + 2 * H, D, generator=g).to(torch.bfloat16)
        x = qkv.to(DEV)
        q, k, v = x[:, :G * H], x[:, G * H:G * H + H], x[:, G * H + H:]
        plan = fa.fa_cache_plan(self.pool, self.table, self.lens, i32(new), PAGE, T)
        before = x.clone()
        fa.fa_rope(q, k, self.rope, plan.positions, q_out=q, k_out=k)
        fa.fa_cache4_write(self.cache, k, v, plan.slots)
        ring, counts, table, lens = self.state
        table, cu, ends, positions, slots, counts, bad = pages_util.plan(ring, counts, table, lens, new, PAGE, T)
        assert not bad and plan.slots.tolist() == slots and plan.ends.tolist() == ends and plan.cu_seqlens.tolist() == cu
        # the turned rows within their bound, and the padded ones as they were
        pos = torch.tensor(positions)[None]
        for got, was in ((q, before[:, :G * H]), (k, before[:, G * H:G * H + H])):
            y, mag = turn(was.cpu().transpose(0, 1)[None], [int(t) for t in self.rope.turns.cpu()], False, self.rope.factor, pos)
            assert ((got.cpu().double().transpose(0, 1)[None] - y).abs() <= bound(y, mag, torch.bfloat16)).all()
        if pad:
            assert torch.equal(x[sum(new):], before[sum(new):])
        # what was written is the code of the rows as the GPU turned them
        self.ref.write(k.cpu(), v.cpu(), slots)
        self.state = (ring, counts, table, ends)
        return plan, q, cu

    def attend(self, plan, q, cu, Nq):
        """The last Nq tokens of every sequence, causal; q as [B, heads, Nq, D] by a view where all bring Nq tokens."""
        B = len(cu) - 1
        rows = q[:B * Nq].unflatten(0, (B, Nq)).transpose(1, 2)
        o, lse = fa.fa_decode_cache4(rows, self.cache, self.table, plan.ends, causal=True)
        table = torch.tensor(self.state[2], dtype=torch.int32)
        within(o, lse, attend_bounds(self.ref, rows.cpu(), table, self.state[3], D ** -0.5, True))

    def trim(self, plan, keep):
        ring, counts, table, ends = self.state
        fa.fa_cache_trim(self.pool, self.table, plan.ends, i32(keep), PAGE)
        ring, counts, bad = pages_util.trim(ring, counts, table, ends, keep, PAGE)
        assert not bad and self.pool.ring.tolist() == ring and self.pool.counts.tolist() == counts
        self.state = (ring, counts, table, list(keep))
        self.lens = i32(keep)


def test_serving_loop():
    rng = random.Random(0)
    B = 5
    s = Server(B, 40, 12)
    plan, q, cu = s.step([30, 1, 0, 77, 16], 4, 1)            # prompts
    s.lens = plan.ends
    # the prompts' prefix in 16 bits is the codes' value, for causal attention over the padded batch
    k, v = fa.fa_cache4_read(s.cache, s.table, s.lens, 80)
    want = s.ref.read(torch.tensor(s.state[2]), s.state[3], 80, torch.bfloat16)
    assert torch.equal(k.cpu(), want[0]) and torch.equal(v.cpu(), want[1])
    o, _ = fa.fa_fwd(k, k, v, causal=True)
    assert torch.isfinite(o).all()
    for step in range(6):                                     # speculative steps of three tokens
        plan, q, cu = s.step([3] * B, step % 2, 10 + step)
        s.attend(plan, q, cu, 3)
        s.trim(plan, [e - rng.randrange(3) for e in s.state[3]])
    s.trim(plan._replace(ends=s.lens), [0, s.state[3][1], s.state[3][2], 0, 5])   # two are done, one is cut
    plan, q, cu = s.step([40, 3, 3, 40, 20], 0, 99)           # their pages serve others
    s.lens = plan.ends
    plan, q, cu = s.step([1] * B, 0, 100)
    s.attend(plan, q, cu, 1)
    assert fa.fa_last_device_status(torch.cuda.current_stream().cuda_stream) == 0


def test_a_refused_sequence_changes_nothing():
    """Without pages its rows go nowhere, and the others are served as if it were not there."""
    s = Server(3, 4, 6)
    plan, q, cu = s.step([10, 50, 3], 0, 1)
    assert plan.ends.tolist() == [10, 0, 0] and s.pool.counts.tolist() == [1, 4]
    s.lens = plan.ends
    plan, q, cu = s.step([1, 1, 1], 0, 2)
    s.attend(plan, q, cu, 1)
    assert fa.fa_last_device_status(torch.cuda.current_stream().cuda_stream) == 0


def test_captured_step():
    """Plan, turn, write, attend and go on, captured once and replayed: the same as the calls one by one."""
    B = 4
    outs = []
    for captured in (False, True):
        torch.manual_seed(0)
        pool, cache = fa.FAPagePool.full(30), fa.FACache4(torch.zeros(30, H, PAGE, D // 8 * 9, dtype=torch.uint8, device=DEV))
        table, lens, new = torch.full((B, 6), -1, dtype=torch.int32, device=DEV), i32([0, 14, 0, 31]), i32([1] * B)
        first = fa.fa_cache_plan(pool, table, i32([0] * B), lens, PAGE, 45)
        x = torch.randn(45, 2, H, D, device=DEV, dtype=torch.bfloat16)
        fa.fa_cache4_write(cache, x[:, 0], x[:, 1], first.slots)
        rope = fa.FARope.new(D)
        steps = torch.randn(20, B, G * H + 2 * H, D, device=DEV, dtype=torch.bfloat16)
        qkv = steps[0].clone()
        seen = []

        def step():
            plan = fa.fa_cache_plan(pool, table, lens, new, PAGE, B)
            q, k = fa.fa_rope(qkv[:, :G * H], qkv[:, G * H:G * H + H], rope, plan.positions)
            fa.fa_cache4_write(cache, k, qkv[:, G * H + H:], plan.slots)
            o, lse = fa.fa_decode_cache4(q[:, :, None], cache, table, plan.ends)
            lens.copy_(plan.ends)
            return o, lse

        if captured:
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                result = step()
        for x in steps:
            qkv.copy_(x)
            if captured:
                graph.replay()
                seen.append([t.clone() for t in result])
            else:
                seen.append([t.clone() for t in step()])
        torch.cuda.synchronize()
        outs.append((seen, lens.tolist(), table.clone(), cache.data.clone()))
    for a, b in zip(*(x[0] for x in outs)):
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    assert outs[0][1] == outs[1][1] == [20, 34, 20, 51]
    assert torch.equal(outs[0][2], outs[1][2]) and torch.equal(outs[0][3], outs[1][3])
