"""What a block and its shared expert keep from the forward to the backward: the
calls that would take another forward's factors, or leave the expert out, are
refused before anything runs, and those that may repeat give the same bits."""
import pytest
import torch

from _gpu_util import DEV

pytestmark = pytest.mark.gpu
BF = torch.bfloat16
T, d, N, K, h, hs = 100, 64, 4, 2, 64, 72


@pytest.fixture(scope="module")
def moe():
    import __graft_entry__
    __graft_entry__.build()
    import combine_expert_gemm_gb300 as m
    return m


@pytest.fixture
def block(moe):
    g = torch.Generator().manual_seed(3)
    r = lambda *q, std=0.1, dt=torch.float32: (torch.randn(*q, generator=g) * std).to(dt).to(DEV)
    s = moe.Shape(T, d, N, K, h, moe.capacity(T, K, N, 5, 4))

    class Block:
        w = [1 + r(d), r(d), r(N, d), r(N), r(N, h, d, dt=BF), r(N, h, d, dt=BF), r(N, d, h, dt=BF)]
        x, dout = r(T, d, std=1.0, dt=BF), r(T, d, std=1.0, dt=BF)
        scale = torch.rand(T, generator=g).to(DEV)
        sc = moe.BlockScratch(s, DEV)

        def state(self):
            return moe.BlockState(s, DEV)

        def expert(self, tokens=T, width=d):
            return moe.SharedExpert(tokens, r(hs, width, dt=BF), r(hs, width, dt=BF), r(width, hs, dt=BF))

        def forward(self, st, **kw):
            return moe.block_forward(st, self.sc, self.x, None, *self.w, **kw).clone()

        def backward(self, st, **kw):
            dx = torch.full((T, d), 7.0, dtype=BF, device=DEV)
            moe.block_backward(st, self.sc, self.dout, dx, torch.ones(2, device=DEV), *self.w, **kw)
            return dx

    return Block()


def test_a_refused_forward_leaves_nothing_saved(moe, block):
    """Its token scale has taken the place of the last forward's: neither is used."""
    e, y, dx = block.expert(), torch.empty(T, d, dtype=BF, device=DEV), torch.empty(T, d, dtype=BF, device=DEV)
    e.forward(block.x, None, y, block.scale)
    with pytest.raises(ValueError):
        e.forward(block.x, None, y[:5], 2 * block.scale)
    with pytest.raises(RuntimeError):
        e.backward(block.x, block.dout, None, dx)
    e.forward(block.x, None, y, block.scale)
    for bad in (block.scale[:5], block.scale.cpu()):
        with pytest.raises(ValueError):
            e.forward(block.x, None, y, bad)  # refused before anything is kept
    e.backward(block.x, block.dout, None, dx)
    torch.cuda.synchronize()
