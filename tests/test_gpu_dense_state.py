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


def test_backward_takes_the_forwards_expert(block):
    st, e, other = block.state(), block.expert(), block.expert()
    block.forward(st, shared=e)
    with pytest.raises(ValueError, match="not the shared expert"):
        block.backward(st)
    block.forward(block.state(), shared=other)
    with pytest.raises(ValueError, match="not the shared expert"):
        block.backward(st, shared=other)
    first = block.backward(st, shared=e)
    assert torch.equal(block.backward(st, shared=e), first)  # the same forward once more
    block.forward(st)
    with pytest.raises(ValueError, match="without one"):
        block.backward(st, shared=e)
    alone = block.backward(st)
    assert not torch.equal(alone, first)
    block.forward(st, shared=e)
    assert torch.equal(block.backward(st, shared=e), first)
    torch.cuda.synchronize()


def test_a_forward_since_is_seen(moe, block):
    a, b, e = block.state(), block.state(), block.expert()
    block.forward(a, shared=e)
    block.forward(b, shared=e)
    with pytest.raises(RuntimeError, match="another forward"):
        block.backward(a, shared=e)
    first = block.backward(b, shared=e)
    block.forward(a, shared=e)  # one after the other, both may use it
    assert torch.equal(block.backward(a, shared=e), first)
    y = torch.empty(T, d, dtype=BF, device=DEV)
    e.forward(block.x, None, y)
    with pytest.raises(RuntimeError, match="another forward"):
        block.backward(a, shared=e)
    e.backward(block.x, block.dout, None, torch.empty_like(y))  # its own, of that forward
    torch.cuda.synchronize()


def test_block_forward_refuses_before_it_runs(moe, block):
    st, e = block.state(), block.expert()
    block.forward(st, shared=e, shared_scale=block.scale)
    first = block.backward(st, shared=e)
    for bad in (dict(shared_scale=block.scale), dict(shared=block.expert(tokens=T + 1)),
                dict(shared=block.expert(width=2 * d)), dict(shared=e, shared_scale=block.scale[:5])):
        with pytest.raises(ValueError):
            block.forward(st, **bad)
    with pytest.raises(TypeError):
        block.forward(st, shared=e, shared_scale=block.scale.double())
    assert torch.equal(block.backward(st, shared=e), first)  # the state is the first forward's still
    torch.cuda.synchronize()


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


def test_captured_blocks_with_a_shared_expert(moe, block):
    """Forward and backward of two blocks, each with its expert, in one graph."""
    states, experts = [block.state(), block.state()], [block.expert(), block.expert()]
    out = [torch.zeros(T, d, dtype=BF, device=DEV) for _ in range(2)]
    dlosses = torch.ones(2, device=DEV)

    def step():
        for st, e in zip(states, experts):
            moe.block_forward(st, block.sc, block.x, None, *block.w, shared=e, shared_scale=block.scale)
        for st, e, o in zip(reversed(states), reversed(experts), out):
            moe.block_backward(st, block.sc, block.dout, o, dlosses, *block.w, shared=e)

    step()
    want = [o.clone() for o in out]
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for o in out:
        o.zero_()
    graph.replay()
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(out, want))
