"""Trains two pre-norm routed-expert blocks for a few steps on one GPU.

    python examples/train_block.py

Each block is layer norm -> routed-expert layer -> residual add (folded into the
next norm), with the balance loss and the z loss on its router; what a block
keeps for its backward is held in 8 bits, and one set of bf16 buffers serves
both.  The task is synthetic: the blocks learn a fixed random linear map of the
tokens.  The routers start biased towards few experts, so the balance loss has
something to do."""
import math
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import combine_expert_gemm_gb300 as moe  # noqa: E402


class Block:
    def __init__(self, shape, gen, dev):
        T, d, N, h = shape.T, shape.d, shape.N, shape.h
        n = lambda *s, std: torch.randn(*s, generator=gen, device=dev) * std
        self.state = moe.BlockState(shape, dev)
        self.gamma, self.beta = torch.ones(d, device=dev), torch.zeros(d, device=dev)
        self.w_router = n(N, d, std=0.02)
        self.bias = torch.linspace(1.5, -1.5, N, device=dev)    # a skewed start
        # fp32 master weights and the bf16 copies that the layer reads
        self.master = [n(N, h, d, std=d ** -0.5), n(N, h, d, std=d ** -0.5), n(N, d, h, std=h ** -0.5)]
        self.experts = [w.to(torch.bfloat16) for w in self.master]
        self.params = self.master + [self.w_router, self.bias, self.gamma, self.beta]

    def forward(self, sc, x, add):
        return moe.block_forward(self.state, sc, x, add, self.gamma, self.beta, self.w_router,
                                 self.bias, *self.experts)

    def backward(self, sc, dh, dlosses, adam):
        moe.block_backward(self.state, sc, dh, dh, dlosses, self.gamma, self.beta, self.w_router,
                           self.bias, *self.experts)
        b = sc.bwd
        # the scratch holds one block's gradients at a time: step before the next block's
        for w, g in zip(self.params, [b.dw_gate, b.dw_up, b.dw_down, b.dw_router, b.dbias, sc.dgamma,
                                      sc.dbeta]):
            w.grad = g
        adam.step()
        for w, c in zip(self.master, self.experts):
            c.copy_(w)


def train(steps=30, T=2048, d=256, N=16, K=2, h=256, lr=1e-2, balance=1.0, z=1e-3, seed=0):
    """Returns the task loss and the blocks' mean balance loss of every step."""
    dev = torch.device("cuda:0")
    gen = torch.Generator(device=dev).manual_seed(seed)
    shape = moe.Shape(T, d, N, K, h, moe.capacity(T, K, N, 2))
    blocks = [Block(shape, gen, dev) for _ in range(2)]
    sc = moe.BlockScratch(shape, dev)
    target_map = torch.randn(d, d, generator=gen, device=dev) * d ** -0.5
    dlosses = torch.tensor([balance, z], device=dev)
    adam = [torch.optim.Adam(blk.params, lr=lr) for blk in blocks]
    task, even = [], []
    for _ in range(steps):
        x = torch.randn(T, d, generator=gen, device=dev).to(torch.bfloat16)
        h, y = x, None
        for blk in blocks:
            y = blk.forward(sc, h, y)
            h = blk.state.h
        err = h.float() + y.float() - x.float() @ target_map
        dh = (err * (2.0 / (T * math.sqrt(d)))).to(torch.bfloat16)  # of sum(err^2) / (T sqrt d)
        for blk, opt in zip(reversed(blocks), reversed(adam)):
            blk.backward(sc, dh, dlosses, opt)
        task.append(err.square().mean())
        even.append(torch.stack([blk.state.losses[0] for blk in blocks]).mean())
    return torch.stack(task).tolist(), torch.stack(even).tolist(), blocks, sc


def held_bytes(obj):
    return sum(t.numel() * t.element_size() for t in vars(obj).values() if isinstance(t, torch.Tensor))


if __name__ == "__main__":
    task, even, blocks, sc = train()
    for i in range(0, len(task), 5):
        print(f"step {i:3d}  task loss {task[i]:.4f}  balance loss {even[i]:.4f}")
    f = sc.fwd
    bf16 = sum(t.numel() * 2 for t in (f.x_disp, f.h_act, f.g_save, f.u_save, f.y_disp))
    print(f"kept per block: {held_bytes(blocks[0].state) / 1e6:.1f} MB "
          f"(the experts' bf16 buffers alone: {bf16 / 1e6:.1f} MB)")
