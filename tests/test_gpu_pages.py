"""fa_cache_plan and fa_cache_trim on the GPU, compared for equality with the definition."""
import random

import pytest
import torch

import attention_forward_02_gb300 as fa
import pages_util

pytestmark = pytest.mark.gpu
DEV = "cuda"


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def status():
    return fa.fa_last_device_status(torch.cuda.current_stream().cuda_stream)


class Batch:
    """Sequences of `lens` tokens, their pages scattered over a pool with `free` pages left in a ring that has gone
    round a few times."""

    def __init__(self, lens, page, free, wide, seed=0, width=0):
        rng = random.Random(seed)
        held = sum(pages_util.pages(n, page) for n in lens if n > 0)
        self.page, self.lens, size = page, lens, max(1, held + free)
        numbers = list(range(size))
        rng.shuffle(numbers)
        self.table = [[-1] * wide for _ in lens]
        for b, n in enumerate(lens):
            for at in range(min(wide, pages_util.pages(n, page)) if n > 0 else 0):
                self.table[b][at] = numbers.pop()
        self.taken = rng.randrange(5 * size)
        self.ring = [-5] * size
        for i in range(free):
            self.ring[(self.taken + i) % size] = numbers.pop(0)
        self.counts = [self.taken, self.taken + free]
        big = torch.full((len(lens), wide + width), -9, dtype=torch.int32)
        big[:, :wide] = torch.tensor(self.table, dtype=torch.int32).reshape(len(lens), wide)
        self.wide_table = big.to(DEV)
        self.gpu_table = self.wide_table[:, :wide]
        self.pool = fa.FAPagePool(i32(self.ring), torch.tensor(self.counts, device=DEV))

    def plan(self, new, T, **kw):
        want = pages_util.plan(self.ring, self.counts, self.table, self.lens, new, self.page, T)
        got = fa.fa_cache_plan(self.pool, self.gpu_table, i32(self.lens), i32(new), self.page, T, **kw)
        self.same(got, want)
        assert status() == (6 if want[-1] else 0)
        self.table, self.ends, self.counts = want[0], want[2], want[5]
        return got, want

    def same(self, got, want):
        assert got.cu_seqlens.tolist() == want[1]
        assert got.ends.tolist() == want[2]
        assert got.positions.tolist() == want[3]
        assert got.slots.tolist() == want[4]
        assert self.gpu_table.tolist() == want[0]
        assert (self.wide_table[:, self.gpu_table.shape[1]:] == -9).all()
        assert self.pool.ring.tolist() == self.ring
        assert self.pool.counts.tolist() == want[5]

    def trim(self, lens, keep):
        ring, counts, bad = pages_util.trim(self.ring, self.counts, self.table, lens, keep, self.page)
        fa.fa_cache_trim(self.pool, self.gpu_table, i32(lens), i32(keep), self.page)
        assert self.pool.ring.tolist() == ring and self.pool.counts.tolist() == counts
        assert self.gpu_table.tolist() == self.table
        assert status() == (6 if bad else 0)
        self.ring, self.counts = ring, counts


@pytest.mark.parametrize("page", [16, 32, 64, 128])
@pytest.mark.parametrize("B", [1, 2, 37, 511, 512, 513, 1500])
def test_mixed(page, B):
    """Lengths of 0, 1, whole pages and others; no, one and many new tokens; rows behind the last sequence."""
    rng = random.Random(B * page)
    lens = [rng.choice([0, 1, page - 1, page, page + 1, rng.randrange(5 * page)]) for _ in range(B)]
    new = [rng.choice([0, 0, 1, 1, 2, page, page + 1, rng.randrange(3 * page)]) for _ in range(B)]
    b = Batch(lens, page, sum(pages_util.pages(n, page) for n in new) + B, 10, seed=B, width=3)
    b.plan(new, sum(new) + rng.randrange(9))
    keep = [rng.randint(n, e) for n, e in zip(lens, b.ends)]
    b.trim(b.ends, keep)
    b.trim(keep, [0 if i % 3 else n for i, n in enumerate(keep)])


@pytest.mark.parametrize("T,pad", [(1, 0), (3, 0), (4, 3), (8191, 0), (16384, 1), (16385, 0), (70001, 6)])
def test_one_prompt(T, pad):
    """A prompt alone, and between sequences with nothing to do."""
    for lens, new in (([0], [T]), ([5, 33, 7], [0, T, 0]), ([0, 0, 64, 0], [0, 0, T, 0])):
        b = Batch(lens, 64, T // 64 + 3, T // 64 + 4, seed=T)
        b.plan(new, T + pad)


def test_largest_batch():
    B = 16384
    rng = random.Random(7)
    lens, new = [rng.randrange(40) for _ in range(B)], [rng.choice([0, 1, 1, 3]) for _ in range(B)]
    b = Batch(lens, 16, B, 4)
    b.plan(new, sum(new) + 5)
    b.trim(b.ends, [rng.randint(0, e) for e in b.ends])


@pytest.mark.parametrize("free", [0, 1, 2, 3, 5, 6, 7, 100])
def test_pool_too_small(free):
    """Served in order while the pages last; sequences that need none are served all the same."""
    lens, new = [10, 16, 0, 31, 5, 16, 0], [3, 1, 40, 1, 20, 0, 1]
    b = Batch(lens, 16, free, 6)
    b.plan(new, sum(new))
    b.trim([max(x, 0) for x in b.ends], [0] * len(lens))


@pytest.mark.parametrize("lens,new,T", [
    ([-1, 5], [4, 4], 8), ([5, 5, 5], [4, -3, 2], 10), ([5, 5], [4, 60], 64), ([5, 64, 5], [2, 1, 3], 6),
    ([5, 5, 5], [4, 4, 4], 7), ([5, 5, 5, 6], [4, 4, 4, 0], 8), ([0, 70, 1], [1, 0, 1], 2), ([3], [2], 0),
    ([2 ** 31 - 1, 1], [2 ** 31 - 1, 3], 9), ([1, 1, 1], [2 ** 31 - 1, 2 ** 31 - 1, 2], 12),
], ids=str)
def test_lengths_that_are_none(lens, new, T):
    """Negative, beyond the page table (4 pages of 16), beyond the rows: refused and reported, the others served."""
    held = [n if 0 <= n <= 64 else 0 for n in lens]
    b = Batch(held, 16, 20, 4)
    b.lens = lens
    want = pages_util.plan(b.ring, b.counts, b.table, lens, [min(n, 2 ** 20) for n in new], 16, T)
    if max(new) < 2 ** 20:
        b.plan(new, T)
    else:  # sums of rows beyond 32 bits: the rows that there are, and their sequences, all the same
        got = fa.fa_cache_plan(b.pool, b.gpu_table, i32(lens), i32(new), 16, T)
        assert got.positions.tolist() == want[3] and got.slots.tolist() == want[4] and got.ends.tolist() == want[2]
        assert got.cu_seqlens.tolist()[-1] == min(2 ** 31 - 1, sum(max(0, n) for n in new))
        assert status() == 6


@pytest.mark.parametrize("counts", [[-1, 3], [5, 4], [0, 1000], [2 ** 62, 2 ** 62 - 1]])
def test_counts_that_are_none(counts):
    b = Batch([5, 16], 16, 4, 4)
    b.counts = counts
    b.pool.counts.copy_(torch.tensor(counts))
    b.plan([3, 1], 4)
    b.trim([5, 16], [5, 0])


def test_table_without_pages():
    """A place below the end that holds no page: its rows have a position and no slot."""
    b = Batch([20, 20], 16, 4, 4)
    for bad in (-1, 10 ** 6):
        b.table[0][1] = bad
        b.gpu_table[0, 1] = bad
        want = pages_util.plan(b.ring, b.counts, b.table, b.lens, [2, 2], 16, 4)
        out = torch.zeros(2, dtype=torch.int64, device=DEV)
        plan = fa.fa_cache_plan(b.pool, b.gpu_table, i32(b.lens), i32([2, 2]), 16, 4, counts=out)
        assert plan.slots.tolist() == want[4] and want[4][:2] == [-1, -1] and want[4][2] >= 0
        assert plan.positions.tolist() == [20, 21, 20, 21]
        assert status() == 6


def test_trim_twice_and_wrong_lengths():
    b = Batch([40, 33, 16], 16, 2, 4)
    b.trim([40, 33, 16], [41, -1, 16])     # longer than it is, negative, nothing to give
    b.trim([40, 33, 16], [0, 0, 0])        # all of it: the ring is full
    b.trim([40, 33, 16], [0, 0, 0])        # again: no room
    b = Batch([40], 16, 2, 4)
    b.trim([65], [0])                      # behind the table
    b.table[0][1] = -3
    b.gpu_table[0, 1] = -3
    b.trim([40], [0])                      # a place without a page goes back as it is


def test_pool_stays_for_another_plan():
    b = Batch([5, 16], 16, 4, 4)
    out = torch.zeros(2, dtype=torch.int64, device=DEV)
    lens = i32(b.lens)
    fa.fa_cache_plan(b.pool, b.gpu_table, lens, i32([30, 9]), 16, 39, counts=out)
    assert out.tolist() == [b.counts[0] + 3, b.counts[1]] and b.pool.counts.tolist() == b.counts
    b.table = b.gpu_table.tolist()
    b.plan([1, 1], 2)


def test_given_outputs_empty_batch_and_full_pool():
    b = Batch([5, 16, 3], 16, 4, 4)
    buf = torch.full((64,), 77, dtype=torch.int32, device=DEV)
    plan = fa.FAPlan(buf[1:5], buf[9:12], buf[17:24], buf[33:40])  # rows that are not 16-byte aligned
    got, _ = b.plan([2, 1, 4], 7, plan=plan)
    assert got is plan
    rest = torch.ones(64, dtype=torch.bool)
    for lo, hi in ((1, 5), (9, 12), (17, 24), (33, 40)):
        rest[lo:hi] = False
    assert (buf.cpu()[rest] == 77).all()
    none = torch.zeros((0, 4), dtype=torch.int32, device=DEV)
    plan = fa.fa_cache_plan(b.pool, none, i32([]), i32([]), 16, 3)
    assert plan.cu_seqlens.tolist() == [0] and plan.slots.tolist() == [-1] * 3 and plan.ends.numel() == 0
    fa.fa_cache_trim(b.pool, none, i32([]), i32([]), 16)
    pool = fa.FAPagePool.full(6)
    table = torch.zeros((1, 8), dtype=torch.int32, device=DEV)
    plan = fa.fa_cache_plan(pool, table, i32([0]), i32([90]), 16, 90)
    assert table.tolist() == [[0, 1, 2, 3, 4, 5, 0, 0]] and pool.counts.tolist() == [6, 6]
    assert status() == 0


def test_graph_replays_a_loop():
    """Steps captured once: lengths, table and pool go on from replay to replay, on two graphs in turn."""
    B, page = 6, 16
    b = Batch([3, 15, 16, 0, 40, 7], page, 60, 8)
    lens, new, keep = i32(b.lens), i32([4] * B), i32([0] * B)
    graphs, plans = [], []
    for _ in range(2):
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            plan = fa.fa_cache_plan(b.pool, b.gpu_table, lens, new, page, 4 * B)
            keep.copy_(lens)
            keep.add_(1)
            fa.fa_cache_trim(b.pool, b.gpu_table, plan.ends, keep, page)
            lens.copy_(keep)
        graphs.append(g)
        plans.append(plan)
    for step in range(10):
        graphs[step % 2].replay()
        torch.cuda.synchronize()
        want = pages_util.plan(b.ring, b.counts, b.table, b.lens, [4] * B, page, 4 * B)
        got = plans[step % 2]
        assert got.slots.tolist() == want[4] and got.ends.tolist() == want[2] and got.cu_seqlens.tolist() == want[1]
        b.table = want[0]
        b.lens = [n + 1 for n in b.lens]
        b.ring, b.counts, _ = pages_util.trim(b.ring, want[5], b.table, want[2], b.lens, page)
        assert b.pool.ring.tolist() == b.ring and b.pool.counts.tolist() == b.counts and lens.tolist() == b.lens
    assert status() == 0


def test_serves_the_8_bit_cache():
    """The plan's cu_seqlens and ends are what fa_cache_write and fa_decode_cache take, its slots where rows went."""
    H, d, page = 2, 64, 16
    pool = fa.FAPagePool.full(20)
    cache = fa.FACache.empty(20, H, page, d)
    table = torch.full((3, 6), -1, dtype=torch.int32, device=DEV)
    lens = i32([0, 0, 0])
    for new in ([20, 0, 7], [1, 33, 1]):
        T = sum(new)
        plan = fa.fa_cache_plan(pool, table, lens, i32(new), page, T)
        x = torch.randn(T, 2, H, d, device=DEV, dtype=torch.bfloat16)
        fa.fa_cache_write(cache, x[:, 0], x[:, 1], table, lens, cu_seqlens=plan.cu_seqlens)
        lens = plan.ends
        codes = cache.k[plan.slots.long() // page, :, plan.slots.long() % page].float()
        back = codes * cache.k_scale[plan.slots.long() // page][..., None]
        assert (back - x[:, 0].float()).abs().max() <= 2.0 ** -4 * x[:, 0].float().abs().max()
    assert lens.tolist() == [21, 33, 8] and status() == 0
