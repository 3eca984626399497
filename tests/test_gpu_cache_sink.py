"""An attention sink, a key that has nearly all of a row's weight and a value of zero: the output is made of the
small weights, which have to keep their bits beside the large one."""
import pytest
import torch

from cache_bounds import attend_bounds, excess, sink
from cache_util import DTYPES, Ref, pages_for

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("n", [500, 4096])
@pytest.mark.parametrize("d,G", [(128, 4), (64, 8), (128, 12), (128, 40)])
def test_sink(fmt, dtype, n, d, G):
    import attention_forward_02_gb300 as fa
    for mass in (0.9, 0.99, 0.999, 0.9999):
        table, pool = pages_for([n], 64, 1)
        ref = Ref(pool, 1, 64, d, fmt, 2)
        if fmt == "int8":  # codes of up to 127 to e4m3's size
            ref.k = (ref.k / 8).round()
        ref.k_scale[:] = 2.0 ** -5
        q = torch.zeros(1, G, 1, d, dtype=DTYPES[dtype])
        sink(ref, table, [n], q, 3, mass)
        got = fa.fa_decode_cache(q.cuda(), ref.to("cuda"), table.cuda(), torch.tensor([n], dtype=torch.int32).cuda())
        want = attend_bounds(ref, q, table, [n], d ** -0.5, False)
        over, lse_over = excess(got[0].double().cpu(), got[1].double().cpu(), want)
        assert over <= 0 and lse_over <= 0, "mass %g: o %.3g, lse %.3g of its bound over it" % (mass, over, lse_over)
