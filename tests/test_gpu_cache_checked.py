"""The checked build over every page size and head dimension: copies of 512 bytes (pages of 16 at d = 32, and the
narrow part at d = 96) up to 8 KB are checked with their own size."""
import pytest
import torch

from cache_bounds import attend_bounds, excess
from cache_util import Ref, pages_for

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
@pytest.mark.parametrize("d", [32, 64, 96, 128])
@pytest.mark.parametrize("page", [16, 64, 128])
def test_page_sizes(monkeypatch, fmt, d, page):
    import attention_forward_02_gb300 as fa
    from attention_forward_02_gb300 import _lib
    chk = _lib.load_checked()
    monkeypatch.setattr(_lib, "_lib", chk)
    stream = torch.cuda.current_stream().cuda_stream
    chk.fa_last_device_status(stream)
    lens = [1100, 1, 0, 77]  # a ring's slots all used, and more than once
    table, pool = pages_for(lens, page, 1)
    ref = Ref(pool, 2, page, d, fmt, 2)
    q = torch.randn(4, 6, 2, d, generator=torch.Generator().manual_seed(3)).half()
    n = torch.tensor(lens, dtype=torch.int32).cuda()
    o, lse = fa.fa_decode_cache(q.cuda(), ref.to("cuda"), table.cuda(), n, causal=True)
    assert fa.fa_last_device_status(stream) == 0
    want = attend_bounds(ref, q, table, lens, d ** -0.5, True)
    over, lse_over = excess(o.double().cpu(), lse.double().cpu(), want)
    assert over <= 0 and lse_over <= 0
