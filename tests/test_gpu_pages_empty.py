"""A plan and a trim of no sequences: the counts that a caller asked for are the pool's, and a plan that was used before
holds no slots of its last step."""
import pytest
import torch

import attention_forward_02_gb300 as fa

pytestmark = pytest.mark.gpu
DEV = "cuda"


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


@pytest.fixture(params=["module", "ctypes"])
def way(request, monkeypatch):
    if request.param == "ctypes":
        monkeypatch.setattr("attention_forward_02_gb300.pages._quick", lambda: False)


def used_pool():
    pool = fa.FAPagePool.full(9)
    pool.counts.copy_(torch.tensor([3, 10]))
    return pool, torch.zeros((0, 4), dtype=torch.int32, device=DEV)


@pytest.mark.parametrize("T", [0, 3, 5000])
@pytest.mark.parametrize("given", [False, True])
@pytest.mark.parametrize("counts", [False, True])
@pytest.mark.parametrize("other", [False, True])
def test_plan(way, T, given, counts, other):
    pool, table = used_pool()
    plan = None
    if given:
        plan = fa.FAPlan(*(torch.full((n,), 77, dtype=torch.int32, device=DEV) for n in (1, 0, T, T)))
    out = torch.full((2,), -9, dtype=torch.int64, device=DEV) if counts else None
    stream = torch.cuda.Stream() if other else None
    torch.cuda.synchronize()
    got = fa.fa_cache_plan(pool, table, i32([]), i32([]), 16, T, counts=out, plan=plan, stream=stream)
    torch.cuda.synchronize()
    assert got.cu_seqlens.tolist() == [0] and got.ends.numel() == 0
    assert got.positions.tolist() == [-1] * T and got.slots.tolist() == [-1] * T
    assert not given or got is plan
    assert pool.counts.tolist() == [3, 10] and pool.ring.tolist() == list(range(9))
    assert out is None or out.tolist() == [3, 10]


@pytest.mark.parametrize("other", [False, True])
def test_trim(way, other):
    pool, table = used_pool()
    out = torch.full((2,), -9, dtype=torch.int64, device=DEV)
    stream = torch.cuda.Stream() if other else None
    torch.cuda.synchronize()
    fa.fa_cache_trim(pool, table, i32([]), i32([]), 16, counts=out, stream=stream)
    torch.cuda.synchronize()
    assert out.tolist() == [3, 10] and pool.counts.tolist() == [3, 10]
    fa.fa_cache_trim(pool, table, i32([]), i32([]), 16)
    assert pool.counts.tolist() == [3, 10] and pool.ring.tolist() == list(range(9))
