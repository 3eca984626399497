"""What the zeros behind a sequence's end that fa_cache_read writes are good for: they are finite, so that causal
attention, which does not see them, may run over the padded batch; every other call counts them as keys of score 0
and has to be given each sequence cut to its length."""
import math

import pytest
import torch

from cache_util import Ref, pages_for

pytestmark = pytest.mark.gpu


def case(fa):
    lens = [100, 7, 49]
    table, pool = pages_for(lens, 16, 1)
    cache = Ref(pool, 2, 16, 64, "e4m3", 2).to("cuda")
    n = torch.tensor(lens, dtype=torch.int32, device="cuda")
    k, v = fa.fa_cache_read(cache, table.cuda(), n, max(lens), dtype=torch.float16)
    return lens, cache, table.cuda(), n, k, v


def test_causal_attention_over_the_padded_batch():
    import attention_forward_02_gb300 as fa
    lens, _, _, _, k, v = case(fa)
    q = torch.randn(k.shape, generator=torch.Generator().manual_seed(3)).half().cuda()
    o, lse = fa.fa_fwd(q, k, v, causal=True)
    for b, n in enumerate(lens):
        o1, lse1 = fa.fa_fwd(*(x[b:b + 1, :, :n].contiguous() for x in (q, k, v)), causal=True)
        assert torch.equal(o[b, :, :n], o1[0]) and torch.equal(lse[b, :, :n], lse1[0])


def test_decoding_needs_each_sequence_cut_to_its_length():
    """Of equal values the mean is that value whatever the weights, and padding pulls it to zero; the sum over n keys
    of score 0 (a zero query) is n."""
    import attention_forward_02_gb300 as fa
    lens, cache, table, n, k, v = case(fa)
    q = torch.zeros(3, 2, 1, 64, dtype=torch.float16, device="cuda")
    _, whole = fa.fa_decode(q, k, v)
    _, want = fa.fa_decode_cache(q, cache, table, n)
    for b, L in enumerate(lens):
        _, lse = fa.fa_decode(*(x[b:b + 1].contiguous() for x in (q, k[:, :, :L], v[:, :, :L])))
        for got, keys in ((lse, L), (want[b], L), (whole[b], 100)):  # the padded call counts all 100
            assert (got - math.log(keys)).abs().max() <= 2.0 ** -18
