"""The block operators together: a stack of two pre-norm blocks against 64-bit
automatic differentiation, and the training example.

Tolerance of the gradients.  Every stored tensor between two steps is bf16
(half an ulp, 2^-9) and the backward's G, U and y come from 8-bit checkpoints:
a block's step is at most its largest magnitude / 64, about 2.5 standard
deviations of normal data / 64, so an element is off by a uniform error of
0.039 / sqrt(12) = 1.1% of the standard deviation.  H and the SwiGLU's
derivatives take that from G and from U (1.6%), bf16 roundings add a few times
0.2%, and the second block's gradient passes the first's weights once more.
4% in the 2-norm covers it; a wrong or missing term is off by far more."""
import os
import sys

import pytest
import torch

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


def _layer(n, p, st, mask, N):
    """The routed-expert layer of n in 64 bits with the routes of st, and its losses."""
    logits = n @ p["w_router"].t() + p["bias"]
    idx, row = st.topk_idx.cpu().long(), st.route_row.cpu()
    gate = torch.softmax(logits.gather(1, idx), 1) * (row >= 0)
    y = torch.zeros_like(n)
    for k in range(idx.shape[1]):
        for e in range(N):
            t = torch.nonzero((idx[:, k] == e) & (row[:, k] >= 0))[:, 0]
            if len(t) == 0:
                continue
            x = n[t]
            a = torch.nn.functional.silu(x @ p["w_gate"][e].t()) * (x @ p["w_up"][e].t())
            y = y.index_add(0, t, gate[t, k][:, None] * (a @ p["w_down"][e].t()))
    live = torch.ones(len(n), dtype=torch.bool) if mask is None else mask != 0
    tc = int(live.sum())
    f = torch.bincount(idx[live].reshape(-1), minlength=N).to(D) / (tc * idx.shape[1])
    lse = torch.logsumexp(logits[live], 1)
    prob = torch.softmax(logits[live], 1).sum(0) / tc
    return y, torch.stack([N * (f * prob).sum(), (lse ** 2).sum() / tc])


@pytest.mark.parametrize("masked", [False, True])
def test_two_blocks_against_automatic_differentiation(moe, masked):
    T, d, N, K, h = 250, 128, 8, 2, 128
    s = moe.Shape(T, d, N, K, h, 80)
    g = torch.Generator().manual_seed(5 + masked)
    r = lambda *q, std=1.0: torch.randn(*q, generator=g) * std
    params = []
    for _ in range(2):
        p = dict(gamma=1 + r(d, std=0.1), beta=r(d, std=0.1), w_router=r(N, d, std=0.1),
                 bias=r(N, std=0.2))
        for n, q in (("w_gate", (N, h, d)), ("w_up", (N, h, d)), ("w_down", (N, d, h))):
            p[n] = r(*q, std=0.1).to(BF)
        params.append(p)
    x = r(T, d).to(BF)
    dout = r(T, d).to(BF)
    mask = (torch.rand(T, generator=g) < 0.8).to(torch.uint8) if masked else None
    # auxiliary weights large enough that their share of the router's gradient shows
    dlosses = torch.tensor([40.0, 5.0])

    sc = moe.BlockScratch(s, DEV)
    states = [moe.BlockState(s, DEV) for _ in range(2)]
    dev = [{k: v.to(DEV) for k, v in p.items()} for p in params]
    hcur, y = x.to(DEV), None
    order = ("gamma", "beta", "w_router", "bias", "w_gate", "w_up", "w_down")
    for st, p in zip(states, dev):
        y = moe.block_forward(st, sc, hcur, y, *(p[k] for k in order),
                              token_mask=None if mask is None else mask.to(DEV))
        hcur = st.h
    out = (hcur.float() + y.float()).cpu()
    dh = dout.to(DEV).clone()
    grads = [None, None]
    for i in (1, 0):
        p = dev[i]
        moe.block_backward(states[i], sc, dh, dh, dlosses.to(DEV), *(p[k] for k in order))
        b = sc.bwd
        grads[i] = dict(gamma=sc.dgamma, beta=sc.dbeta, w_router=b.dw_router, bias=b.dbias,
                        w_gate=b.dw_gate, w_up=b.dw_up, w_down=b.dw_down)
        grads[i] = {k: v.clone().cpu().to(D) for k, v in grads[i].items()}
    torch.cuda.synchronize()
    for ws in (sc.fwd.ffn_ws, sc.bwd.ws, sc.dense_ws):
        assert moe.read_device_error(ws) == 0

    ps = [{k: v.to(D).requires_grad_() for k, v in p.items()} for p in params]
    x64 = x.to(D).requires_grad_()
    hc, aux = x64, 0.0
    for st, p in zip(states, ps):
        c = hc - hc.mean(1, keepdim=True)
        n = c / torch.sqrt((c * c).mean(1, keepdim=True) + 1e-5) * p["gamma"] + p["beta"]
        yy, losses = _layer(n, p, st, mask, N)
        assert torch.allclose(st.losses.cpu().to(D), losses.detach(), rtol=0.03)
        aux = aux + (losses * dlosses.to(D)).sum()
        hc = hc + yy
    off = lambda a, b: ((a - b).norm() / b.norm()).item()
    assert off(out.to(D), hc.detach()) < 0.02
    ((hc * dout.to(D)).sum() + aux).backward()
    assert off(dh.cpu().to(D), x64.grad) < TOL
    for i in range(2):
        for k in order:
            assert off(grads[i][k], ps[i][k].grad) < TOL, (i, k)


def test_train_example_learns_and_balances(moe):
    sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
    import train_block
    task, even, blocks, sc = train_block.train(steps=30)
    assert all(map(lambda v: v == v, task + even))
    assert task[-1] < 0.9 * task[0]
    assert even[-1] < even[0] and even[-1] < 1.5
    f = sc.fwd
    bf16 = sum(t.numel() * 2 for t in (f.x_disp, f.h_act, f.g_save, f.u_save, f.y_disp))
    st = blocks[0].state
    held = sum(t.numel() for t in (st.g_q, st.g_scale, st.u_q, st.u_scale, st.y_q, st.y_scale))
    assert held * 3 < bf16


@pytest.mark.parametrize("xt", [BF, torch.float32])
@pytest.mark.parametrize("side", [False, True])
def test_caller_may_reuse_its_input_and_mask_after_the_forward(moe, xt, side):
    """What the backward needs of the first block's input and of the mask is
    the state's own: a caller who fills the same buffers with the next batch
    before the backward gets the same gradients, bit for bit."""
    T, d, N, K, h = 200, 128, 8, 2, 64
    s = moe.Shape(T, d, N, K, h, 80)
    g = torch.Generator().manual_seed(9)
    r = lambda *q, std=1.0: (torch.randn(*q, generator=g) * std).to(DEV)
    p = [1 + r(d, std=0.1), r(d, std=0.1), r(N, d, std=0.1), r(N, std=0.2)]
    p += [r(N, h, d, std=0.1).to(BF), r(N, h, d, std=0.1).to(BF), r(N, d, h, std=0.1).to(BF)]
    x, dh, dlosses = r(T, d).to(xt), r(T, d).to(BF), torch.tensor([40.0, 5.0], device=DEV)
    mask = (torch.rand(T, generator=g) < 0.7).to(torch.uint8).to(DEV)
    stream = torch.cuda.Stream() if side else None
    runs = []
    for reuse in (False, True):
        st, sc = moe.BlockState(s, DEV), moe.BlockScratch(s, DEV)
        xin, m, dx = x.clone(), mask.clone(), torch.empty(T, d, dtype=BF, device=DEV)
        torch.cuda.synchronize()
        moe.block_forward(st, sc, xin, None, *p, token_mask=m, stream=stream)
        torch.cuda.synchronize()
        assert torch.equal(st.h, x)
        if reuse:
            xin.fill_(3.0)
            m.fill_(1)
            torch.cuda.synchronize()
        moe.block_backward(st, sc, dh, dx, dlosses, *p, stream=stream)
        torch.cuda.synchronize()
        runs.append([t.clone() for t in (dx, sc.dgamma, sc.dbeta, sc.dlogits, sc.bwd.dw_router, sc.bwd.dw_up)])
    for a, b in zip(*runs):
        assert torch.equal(a, b)


def test_block_refuses_an_input_of_another_shape(moe):
    """Fewer rows would leave the rest of the state's rows those of an earlier call."""
    s = moe.Shape(64, 128, 4, 2, 64, 40)
    st, sc = moe.BlockState(s, DEV), moe.BlockScratch(s, DEV)
    w = [torch.ones(128, device=DEV), None, torch.zeros(4, 128, device=DEV), None]
    w += [torch.zeros(*q, dtype=BF, device=DEV) for q in ((4, 64, 128), (4, 64, 128), (4, 128, 64))]
    for q in ((63, 128), (1, 128), (128, 64)):
        with pytest.raises(ValueError):
            moe.block_forward(st, sc, torch.zeros(*q, dtype=BF, device=DEV), None, *w)
