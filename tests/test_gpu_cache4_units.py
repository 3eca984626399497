"""Attention over the 4-bit cache within bounds whose merges are those of its kernels: a part has 128 keys at least
(cache4_util takes 64, the 8-bit cache's smallest unit; a warp that has a whole segment in 32-key stages merges nothing)."""
import pytest
import torch

import attention_forward_02_gb300 as fa
import cache4_util
from cache4_util import DTYPES, Ref, attend_bounds, pages_for, within

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.mark.parametrize("d,H,G,Nq", [(32, 2, 1, 1), (64, 2, 5, 1), (128, 1, 4, 4), (128, 1, 20, 1), (96, 1, 12, 4), (96, 2, 8, 1)])
@pytest.mark.parametrize("lens,page", [([20000, 1, 3000], 32), ([900, 128, 129], 128), ([300] * 300, 16)])
def test_attend(monkeypatch, d, H, G, Nq, lens, page):
    monkeypatch.setattr(cache4_util, "STEP", 128)
    table, pool = pages_for(lens, page, 4)
    ref = Ref(pool, H, page, d, seed=d)
    dtype = DTYPES["fp16" if G % 2 else "bf16"]
    q = torch.randn(len(lens), H * G, Nq, d, generator=torch.Generator().manual_seed(G)).to(dtype)
    o, lse = fa.fa_decode_cache4(q.to(DEV), ref.to(DEV), table.to(DEV), torch.tensor(lens, dtype=torch.int32, device=DEV),
                                 causal=True)
    within(o, lse, attend_bounds(ref, q, table, lens, d ** -0.5, True))
