"""fa_rope in place on query and key rows that lie between one another in one buffer."""
import pytest
import torch

import attention_forward_02_gb300 as fa

pytestmark = pytest.mark.gpu
DEV = "cuda"


def normal(shape, dtype, seed):
    return torch.randn(shape, generator=torch.Generator().manual_seed(seed)).to(dtype).to(DEV)


# how a buffer's query and key rows are cut out of it, and its shape
LAYOUTS = {
    "T H 3 d": (lambda x: (x[:, :, 0], x[:, :, 1]), lambda B, N, H, d: (B * N, H, 3, d)),
    "B N H 3 d": (lambda x: tuple(x[:, :, :, i].transpose(1, 2) for i in range(2)), lambda B, N, H, d: (B, N, H, 3, d)),
    "B H+1 N d": (lambda x: (x[:, :-1], x[:, -1:]), lambda B, N, H, d: (B, H + 1, N, d)),
    "B H N 2 d": (lambda x: (x[:, :, :, 1], x[:, :, :, 0]), lambda B, N, H, d: (B, H, N, 2, d)),
}


@pytest.mark.parametrize("layout", LAYOUTS)
@pytest.mark.parametrize("B,N,H,d", [(2, 5, 3, 64), (3, 1, 20, 32), (2, 700, 8, 128), (1, 33, 1, 96)])
@pytest.mark.parametrize("backward", [False, True])
@pytest.mark.parametrize("quick", [True, False])
def test_in_place(layout, B, N, H, d, backward, quick, monkeypatch):
    if not quick:
        monkeypatch.setattr("attention_forward_02_gb300.rope._quick", lambda: False)
    cut, shape = LAYOUTS[layout]
    rope = fa.FARope.new(d // 2 if d == 64 else d, interleaved=bool(H % 2))
    x = normal(shape(B, N, H, d), torch.bfloat16, d)
    want = x.clone()
    q, k = cut(x)
    pos = (torch.arange(q.shape[0] if q.dim() == 3 else q.shape[2], device=DEV) * 13).int()
    for y, z in zip(cut(want), fa.fa_rope(q, k, rope, pos, backward=backward)):
        y.copy_(z)
    yq, yk = fa.fa_rope(q, k, rope, pos, backward=backward, q_out=q, k_out=k)
    assert yq is q and yk is k
    assert torch.equal(x, want)  # the values' rows among them
