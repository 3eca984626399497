"""The checked build: attention over the 4-bit cache at every page size and head dimension, segments of a block, of
several and of a warp, and the calls around it."""
import pytest
import torch

from cache4_util import Ref, attend_bounds, pages_for, within

pytestmark = pytest.mark.gpu


@pytest.fixture
def checked(monkeypatch):
    from attention_forward_02_gb300 import _lib
    chk = _lib.load_checked()
    monkeypatch.setattr(_lib, "_lib", chk)
    stream = torch.cuda.current_stream().cuda_stream
    chk.fa_last_device_status(stream)
    yield
    assert chk.fa_last_device_status(stream) == 0


@pytest.mark.parametrize("d", [32, 64, 96, 128])
@pytest.mark.parametrize("page", [16, 32, 64, 128])
@pytest.mark.parametrize("G,Nq", [(2, 2), (3, 2), (3, 5), (20, 2)])
def test_attention(checked, d, page, G, Nq):
    import attention_forward_02_gb300 as fa
    for lens in ([1900, 1, 0, 77, 600], [300, 1, 17]):  # a ring's slots all used, and more than once; whole segments
        table, pool = pages_for(lens, page, 1)
        ref = Ref(pool, 2, page, d, 2)
        q = torch.randn(len(lens), 2 * G, Nq, d, generator=torch.Generator().manual_seed(3)).half()
        n = torch.tensor(lens, dtype=torch.int32).cuda()
        o, lse = fa.fa_decode_cache4(q.cuda(), ref.to("cuda"), table.cuda(), n, causal=True)
        within(o, lse, attend_bounds(ref, q, table, lens, d ** -0.5, True))


@pytest.mark.parametrize("d", [32, 64, 96, 128])
@pytest.mark.parametrize("page", [16, 32, 64, 128])
@pytest.mark.parametrize("G,Nq", [(2, 2), (3, 2)])
def test_attention_of_many_segments(checked, d, page, G, Nq):
    import attention_forward_02_gb300 as fa
    lens = [(71 * b) % 257 for b in range(335)]
    table, pool = pages_for(lens, page, 1)
    ref = Ref(pool, 2, page, d, 2)
    q = torch.randn(len(lens), 2 * G, Nq, d, generator=torch.Generator().manual_seed(3)).half()
    n = torch.tensor(lens, dtype=torch.int32).cuda()
    o, lse = fa.fa_decode_cache4(q.cuda(), ref.to("cuda"), table.cuda(), n, causal=True)
    within(o, lse, attend_bounds(ref, q, table, lens, d ** -0.5, True))


def test_around_it(checked):
    import attention_forward_02_gb300 as fa
    pool, table = fa.FAPagePool.full(200), torch.full((3, 80), -1, dtype=torch.int32, device="cuda")
    lens, new = torch.zeros(3, dtype=torch.int32, device="cuda"), torch.tensor([900, 1, 37], dtype=torch.int32, device="cuda")
    for T in (938, 6000):
        plan = fa.fa_cache_plan(pool, table, lens, new, 16, T)
        x = torch.randn(T, 8, 96, device="cuda", dtype=torch.bfloat16)
        q, k = fa.fa_rope(x[:, :4], x[:, 4:6], fa.FARope.new(48), plan.positions)
        cache = fa.FACache4(torch.zeros(200, 2, 16, 108, dtype=torch.uint8, device="cuda"))
        fa.fa_cache4_write(cache, k, x[:, 6:], plan.slots)
        fa.fa_cache4_read(cache, table, plan.ends, 901)
        fa.fa_cache_trim(pool, table, plan.ends, lens, 16)
    assert int(pool.counts[1] - pool.counts[0]) == 200
