"""As many rows as an int counts: fa_cache4_write, one row's values for all of them (stride 0), and fa_cache_plan."""
import pytest
import torch

import attention_forward_02_gb300 as fa
from cache4_util import Ref

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.mark.parametrize("T", [2 ** 31 - 1, 2 ** 31 - 40])
@pytest.mark.parametrize("d", [32, 64])
def test_write(T, d):
    page = 16
    ref = Ref(3, 1, page, d)
    cache = ref.to(DEV)
    k, v = (torch.randn(1, 1, d, generator=torch.Generator().manual_seed(s)).to(torch.bfloat16) for s in (1, 2))
    slots = torch.full((T,), -1, dtype=torch.int32, device=DEV)
    slots[0], slots[T // 2], slots[T - 1] = 7, 20, 47
    fa.fa_cache4_write(cache, k.to(DEV).expand(T, 1, d), v.to(DEV).expand(T, 1, d), slots)
    ref.write(k.expand(3, 1, d), v.expand(3, 1, d), [7, 20, 47])
    assert torch.equal(cache.data.cpu(), ref.bytes())
    assert fa.fa_last_device_status(torch.cuda.current_stream().cuda_stream) == 0


@pytest.mark.parametrize("T", [2 ** 31 - 1, 2 ** 31 - 500])
def test_plan(T):
    pool = fa.FAPagePool.full(9)
    table = torch.full((3, 4), -1, dtype=torch.int32, device=DEV)
    lens, new = (torch.tensor(x, dtype=torch.int32, device=DEV) for x in ([0, 5, 16], [17, 0, 2]))
    plan = fa.fa_cache_plan(pool, table, lens, new, 16, T)
    assert plan.positions[:20].tolist() == list(range(17)) + [16, 17, -1]
    assert plan.slots[:20].tolist() == list(range(17)) + [32, 33, -1]
    for rows in (plan.positions, plan.slots):
        assert rows.shape == (T,) and bool((rows[19:] == -1).all())
    assert fa.fa_last_device_status(torch.cuda.current_stream().cuda_stream) == 0
