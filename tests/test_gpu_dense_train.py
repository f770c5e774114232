"""The dense operators together in a training block: a shared expert beside the
routed ones against 64-bit automatic differentiation and against the single
calls, the training example with both, and Muon over all of a block's matrices.

Tolerance of the gradients: 4% in the 2-norm, as for the blocks without a shared
expert (the experts' buffers come from 8-bit checkpoints, 1.1% each; the shared
expert adds bf16 roundings only, 0.6%)."""
import os
import sys

import pytest
import torch

import _dense_ref as ref
from _gpu_util import DEV

pytestmark = pytest.mark.gpu
D, BF = torch.float64, torch.bfloat16
TOL = 0.04


@pytest.fixture(scope="module")
def moe():
    import __graft_entry__
    __graft_entry__.build()
    import combine_expert_gemm_gb300 as m
    return m


def _setup(moe, T, d, N, K, h, hs, seed):
    s = moe.Shape(T, d, N, K, h, moe.capacity(T, K, N, 5, 4))
    g = torch.Generator().manual_seed(seed)
    r = lambda *q, std=1.0: torch.randn(*q, generator=g) * std
    p = dict(gamma=1 + r(d, std=0.1), beta=r(d, std=0.1), w_router=r(N, d, std=0.1), bias=r(N, std=0.2),
             w_gate=r(N, h, d, std=0.1).to(BF), w_up=r(N, h, d, std=0.1).to(BF), w_down=r(N, d, h, std=0.1).to(BF))
    e = dict(w_gate=r(hs, d, std=0.1).to(BF), w_up=r(hs, d, std=0.1).to(BF), w_down=r(d, hs, std=0.1).to(BF))
    return s, p, e, r(T, d).to(BF), r(T, d).to(BF), torch.rand(T, generator=g)


@pytest.mark.parametrize("scaled,act", [(False, "silu"), (True, "gelu")])
def test_block_with_shared_expert(moe, scaled, act):
    T, d, N, K, h, hs = 250, 128, 8, 2, 128, 200
    s, p, e, x, dout, scale = _setup(moe, T, d, N, K, h, hs, 5)
    dlosses = torch.tensor([40.0, 5.0])
    order = ("gamma", "beta", "w_router", "bias", "w_gate", "w_up", "w_down")
    w = [p[k].to(DEV) for k in order]
    ew = [e[k].to(DEV) for k in ("w_gate", "w_up", "w_down")]
    st, sc = moe.BlockState(s, DEV), moe.BlockScratch(s, DEV)
    shared = moe.SharedExpert(T, *ew, act=act)
    sd = scale.to(DEV) if scaled else None
    y = moe.block_forward(st, sc, x.to(DEV), None, *w, shared=shared, shared_scale=sd).clone()
    if scaled:
        sd.fill_(7.0)  # the backward has its own copy
    dx = dout.to(DEV).clone()
    moe.block_backward(st, sc, dx, dx, dlosses.to(DEV), *w, shared=shared)
    torch.cuda.synchronize()
    assert moe.read_device_error(shared.ws) == 0

    # the single calls give the same bits
    st2, sc2 = moe.BlockState(s, DEV), moe.BlockScratch(s, DEV)
    y2 = moe.block_forward(st2, sc2, x.to(DEV), None, *w)
    o = [torch.empty_like(t) for t in (shared.h_act, shared.p_save, shared.q_save)]
    out = torch.empty_like(y2)
    moe.gated_ffn(st2.n, *ew, y2, scale.to(DEV) if scaled else None, out, *o, shared.ws, act=act)
    assert torch.equal(out, y)
    assert all(torch.equal(a, b) for a, b in zip(o, (shared.h_act, shared.p_save, shared.q_save)))

    # 64 bits
    c = x.to(D).requires_grad_()
    q = {k: v.to(D).requires_grad_() for k, v in p.items()}
    qe = {k: v.to(D).requires_grad_() for k, v in e.items()}
    s64 = scale.to(D).requires_grad_()
    m = c - c.mean(1, keepdim=True)
    n = m / torch.sqrt((m * m).mean(1, keepdim=True) + 1e-5) * q["gamma"] + q["beta"]
    logits = n @ q["w_router"].t() + q["bias"]
    idx, row = st.topk_idx.cpu().long(), st.route_row.cpu()
    gate = torch.softmax(logits.gather(1, idx), 1) * (row >= 0)
    yy = torch.zeros_like(n)
    for k in range(K):
        for i in range(N):
            t = torch.nonzero((idx[:, k] == i) & (row[:, k] >= 0))[:, 0]
            a = torch.nn.functional.silu(n[t] @ q["w_gate"][i].t()) * (n[t] @ q["w_up"][i].t())
            yy = yy.index_add(0, t, gate[t, k][:, None] * (a @ q["w_down"][i].t()))
    f = torch.bincount(idx.reshape(-1), minlength=N).to(D) / (T * K)
    aux = dlosses[0].to(D) * N * (f * torch.softmax(logits, 1).mean(0)).sum()
    aux = aux + dlosses[1].to(D) * (torch.logsumexp(logits, 1) ** 2).mean()
    fn = {"silu": torch.nn.functional.silu, "gelu": lambda v: torch.nn.functional.gelu(v, approximate="tanh")}[act]
    dense = (fn(n @ qe["w_gate"].t()) * (n @ qe["w_up"].t())) @ qe["w_down"].t()
    yy = yy + (dense * s64[:, None] if scaled else dense)
    off = lambda a, b: ((a.cpu().to(D) - b).norm() / b.norm()).item()
    assert off(y, yy.detach()) < 0.02
    (((c + yy) * dout.to(D)).sum() + aux).backward()
    assert off(dx, c.grad) < TOL
    for k in ("w_gate", "w_up", "w_down"):
        assert off(getattr(shared, "d" + k), qe[k].grad) < TOL, k
        assert off(getattr(sc.bwd, "d" + k), q[k].grad) < TOL, k
    assert off(sc.bwd.dw_router, q["w_router"].grad) < TOL
    assert off(sc.dgamma, q["gamma"].grad) < TOL
    if scaled:
        assert off(shared.dtoken_scale, s64.grad) < TOL


def test_shared_expert_refuses(moe):
    w = [torch.zeros(*q, dtype=BF, device=DEV) for q in ((64, 64), (64, 64), (64, 64))]
    e = moe.SharedExpert(10, *w)
    x, y = torch.zeros(10, 64, dtype=BF, device=DEV), torch.zeros(10, 64, dtype=BF, device=DEV)
    with pytest.raises(RuntimeError):
        e.backward(x, y, None, torch.zeros_like(x))
    with pytest.raises(ValueError):
        e.forward(x[:9], None, y)
    with pytest.raises(ValueError):
        e.forward(x, None, y, torch.ones(9, device=DEV))
    with pytest.raises(ValueError):
        moe.Muon([])
    e.forward(x, None, y)
    e.backward(x, y, None, torch.empty_like(x))


def test_block_without_shared_expert_keeps_its_bits(moe):
    s, p, e, x, dout, _ = _setup(moe, 100, 64, 4, 2, 64, 64, 6)
    w = [p[k].to(DEV) for k in ("gamma", "beta", "w_router", "bias", "w_gate", "w_up", "w_down")]
    runs = []
    for kw in ({}, dict(shared=None)):
        st, sc = moe.BlockState(s, DEV), moe.BlockScratch(s, DEV)
        y = moe.block_forward(st, sc, x.to(DEV), None, *w, **kw).clone()
        dx = torch.empty(100, 64, dtype=BF, device=DEV)
        moe.block_backward(st, sc, dout.to(DEV), dx, torch.ones(2, device=DEV), *w, **kw)
        runs.append((y, dx, sc.bwd.dw_gate.clone()))
    assert all(torch.equal(a, b) for a, b in zip(*runs))


def test_muon_over_a_blocks_matrices(moe):
    """Two steps of every matrix of a block, routed and shared, against the formula."""
    T, d, N, K, h, hs = 120, 64, 4, 2, 128, 72
    s, p, e, x, dout, _ = _setup(moe, T, d, N, K, h, hs, 8)
    w = [p[k].to(DEV) for k in ("gamma", "beta", "w_router", "bias", "w_gate", "w_up", "w_down")]
    st, sc = moe.BlockState(s, DEV), moe.BlockScratch(s, DEV)
    shared = moe.SharedExpert(T, *(e[k].to(DEV) for k in ("w_gate", "w_up", "w_down")))
    copies = w[4:] + [shared.w_gate, shared.w_up, shared.w_down]
    master = [c.float() for c in copies]
    opt = moe.Muon(zip(master, copies), lr=0.05, mu=0.9, weight_decay=0.1)
    want = [m.cpu().to(D) for m in master]
    mom = [torch.zeros_like(v) for v in want]
    lr32, mu32, wd32 = (float(torch.tensor(v)) for v in (0.05, 0.9, 0.1))
    for _ in range(2):
        moe.block_forward(st, sc, x.to(DEV), None, *w, shared=shared)
        dx = dout.to(DEV).clone()
        moe.block_backward(st, sc, dx, dx, torch.ones(2, device=DEV), *w, shared=shared)
        grads = [sc.bwd.dw_gate, sc.bwd.dw_up, sc.bwd.dw_down, shared.dw_gate, shared.dw_up, shared.dw_down]
        g64 = [g.cpu().to(D) for g in grads]
        opt.step(grads)
        for i, g in enumerate(g64):
            mom[i] = mu32 * mom[i] + g
            o, _ = ref.newton_schulz((g + mu32 * mom[i]).reshape(-1, *g.shape[-2:]))
            rows, cols = g.shape[-2:]
            want[i] = (1 - lr32 * wd32) * want[i] - lr32 * max(1.0, rows / cols) ** 0.5 * o.reshape(g.shape)
    for m, c, q in zip(master, copies, want):
        # the factors' bound (1e-3 of their norm at these sizes, times lr) and fp32 roundings
        assert float((m.cpu().to(D) - q).norm()) < 1e-4 * float(q.norm())
        assert torch.equal(c, m.to(BF))
    assert moe.read_device_error(opt.ws) == 0
    with pytest.raises(ValueError):
        opt.step(grads[:2])


@pytest.mark.parametrize("muon,shared_h", [(True, 0), (True, 200), (False, 128)])
def test_train_example_runs_with_muon_and_shared_experts(moe, muon, shared_h):
    sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
    import train_block
    task, even, blocks, sc = train_block.train(steps=3, T=512, d=128, N=8, h=64, muon=muon, shared_h=shared_h)
    assert all(v == v for v in task + even)
    for blk in blocks:
        for m, c in zip(blk.master, blk.experts):
            assert bool(m.isfinite().all()) and torch.equal(c, m.to(BF))
        assert (blk.shared is not None) == (shared_h > 0)
