"""The block operators (include/moe_block.h) on the CPU: refusals before
anything is enqueued, and the gradient formulas that the GPU tests use
compared with differences of the 64-bit forward."""
import ctypes

import pytest
import torch

import _block_ref as ref


@pytest.fixture(scope="module")
def moe():
    import __graft_entry__
    __graft_entry__.build()
    import combine_expert_gemm_gb300 as m
    return m


A, MIS = ctypes.c_void_p(4096), ctypes.c_void_p(4096 + 8)
BF, FP = 0, 1


def _shape(moe, **kw):
    base = dict(T=64, d=128, N=8, K=2, h=256, cap=20)
    base.update(kw)
    return ctypes.byref(moe.Shape(**base))


def test_layer_norm_refusals(moe):
    f = moe.lib().moe_layer_norm

    def call(rows=4, d=64, dt=BF, x=A, add=A, gamma=A, beta=A, eps=1e-5, x_sum=A, y=A, mean=A,
             rstd=A):
        return f(rows, d, dt, x, add, gamma, beta, eps, x_sum, y, mean, rstd, None)

    assert call(rows=-1) == 1 and call(d=0) == 1
    assert call(d=12) == 2                               # not a multiple of 8
    assert call(d=16392) == 5                            # wider than the kernels
    assert call(dt=2) == 1 and call(dt=-1) == 1
    for eps in (0.0, -1e-5, float("nan"), float("inf")):
        assert call(eps=eps) == 1
    assert call(x=None) == 1 and call(y=None) == 1
    assert call(add=None) == 1                           # x_sum without add
    assert call(x_sum=None) == 1                         # add without x_sum
    assert call(mean=None) == 1 and call(rstd=None) == 1
    for name in ("x", "add", "gamma", "beta", "x_sum", "y", "mean", "rstd"):
        assert call(**{name: MIS}) == 2, name
    assert call(rows=0, x=None, y=None) == 0             # nothing to do, nothing enqueued


def test_layer_norm_backward_refusals(moe):
    lib = moe.lib()
    need = lib.moe_layer_norm_backward_workspace_bytes(4, 64)
    assert need >= 256
    assert lib.moe_layer_norm_backward_workspace_bytes(-1, 64) == 0
    assert lib.moe_layer_norm_backward_workspace_bytes(4, 12) == 0

    def call(rows=4, d=64, dt=BF, x=A, yt=FP, dy=A, gamma=A, mean=A, rstd=A, gt=BF, dres=A, dx=A,
             dgamma=A, dbeta=A, ws=A, n=need):
        return lib.moe_layer_norm_backward(rows, d, dt, x, yt, dy, gamma, mean, rstd, gt, dres, dx,
                                           dgamma, dbeta, ws, n, None)

    assert call(rows=-1) == 1 and call(d=4) == 2 and call(d=16392) == 5
    assert call(dt=2) == 1 and call(yt=2) == 1 and call(gt=-1) == 1
    for name in ("x", "dy", "mean", "rstd", "dx"):
        assert call(**{name: None}) == 1, name
    for name in ("x", "dy", "gamma", "mean", "rstd", "dres", "dx", "dgamma", "dbeta"):
        assert call(**{name: MIS}) == 2, name
    assert call(n=need - 1) == 3 and call(ws=MIS) == 3 and call(ws=None) == 3


def test_balance_loss_refusals(moe):
    lib, s = moe.lib(), _shape(moe)
    need = lib.moe_balance_loss_workspace_bytes(s)
    assert need >= 256 and lib.moe_balance_loss_workspace_bytes(_shape(moe, K=0)) == 0
    f = [A, A, A, A, A, A, A, A]      # logits, topk_idx, mask, count, tokens, prob, lse, losses
    for i in (0, 1, 3, 4, 5, 6, 7):
        bad = list(f)
        bad[i] = None
        assert lib.moe_balance_loss(s, *bad, A, need, None) == 1, i
    for i in range(8):
        bad = list(f)
        bad[i] = MIS
        assert lib.moe_balance_loss(s, *bad, A, need, None) == 2, i
    assert lib.moe_balance_loss(s, *f, A, need - 1, None) == 3
    assert lib.moe_balance_loss(s, *f, MIS, need, None) == 3
    assert lib.moe_balance_loss(s, *f, None, need, None) == 3
    assert lib.moe_balance_loss(_shape(moe, K=9), *f, A, need, None) == 1

    b = [A] * 9          # logits, topk_idx, mask, count, tokens, lse, dlosses, dlogit, dlogits
    for i in (0, 1, 3, 4, 5, 6, 8):
        bad = list(b)
        bad[i] = None
        assert lib.moe_balance_loss_backward(s, *bad, None) == 1, i
    for i in range(9):
        bad = list(b)
        bad[i] = MIS
        assert lib.moe_balance_loss_backward(s, *bad, None) == 2, i
    assert lib.moe_balance_loss_backward(_shape(moe, T=0), *([None] * 9), None) == 0


def test_router_dense_backward_refusals(moe):
    lib, s = moe.lib(), _shape(moe)
    need = lib.moe_router_dense_backward_workspace_bytes(s)
    assert need >= 256 and lib.moe_router_dense_backward_workspace_bytes(_shape(moe, T=-1)) == 0
    f = [A] * 7                       # x, w_router, dlogits, dx_in, dx, dw_router, dbias
    for i in (0, 1, 2, 4):            # dx_in without dx counts as missing dx
        bad = list(f)
        bad[i] = None
        assert lib.moe_router_dense_backward(s, *bad, A, need, None) == 1, i
    for i in range(7):
        bad = list(f)
        bad[i] = MIS
        assert lib.moe_router_dense_backward(s, *bad, A, need, None) == 2, i
    assert lib.moe_router_dense_backward(s, *f, A, need - 1, None) == 3
    assert lib.moe_router_dense_backward(s, *f, MIS, need, None) == 3
    # nothing asked for: nothing enqueued
    assert lib.moe_router_dense_backward(s, A, A, A, None, None, None, None, A, need, None) == 0


def test_checkpoint_refusals(moe):
    lib, s = moe.lib(), _shape(moe)
    f = [A] * 10                      # offset, g, u, y, then (codes, scales) of each
    for i in (0, 4, 5, 6, 7, 8, 9):
        bad = list(f)
        bad[i] = None
        assert lib.moe_checkpoint_save(s, *bad, None) == 1, i
    for i in range(10):
        bad = list(f)
        bad[i] = MIS
        assert lib.moe_checkpoint_save(s, *bad, None) == 2, i
    for kw in (dict(d=136), dict(h=264)):
        assert lib.moe_checkpoint_save(_shape(moe, **kw), *f, None) == 5
        assert lib.moe_checkpoint_restore(_shape(moe, **kw), *f[:8], None) == 5
        assert lib.moe_combine_backward_checkpoint(_shape(moe, **kw), *f[:8], None) == 5
    assert lib.moe_checkpoint_save(_shape(moe, cap=0), *([None] * 10), None) == 0
    assert lib.moe_checkpoint_save(s, A, *([None] * 9), None) == 0      # every source left out
    for i in range(8):
        bad = [A] * 8
        bad[i] = None
        assert lib.moe_checkpoint_restore(s, *bad, None) == 1, i
        bad[i] = MIS
        assert lib.moe_checkpoint_restore(s, *bad, None) == 2, i
    for i in range(8):                # dy .. dgate, and dlogit, which may be NULL
        bad = [A] * 8
        bad[i] = None
        assert i == 7 or lib.moe_combine_backward_checkpoint(s, *bad, None) == 1, i
        bad[i] = MIS
        assert lib.moe_combine_backward_checkpoint(s, *bad, None) == 2, i
    assert lib.moe_combine_backward_checkpoint(_shape(moe, T=0), *([None] * 8), None) == 0


def test_binding_refuses_wrong_tensors(moe, monkeypatch):
    """Wrong types, sizes and devices raise in the binding, before any call."""
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    x = torch.zeros(4, 64)
    with pytest.raises(ValueError, match="x: must be a CUDA tensor"):
        moe.layer_norm(x, None, None, None, 1e-5, None, x, None, None)
    with pytest.raises(TypeError, match="x: expected a bfloat16 or float32"):
        moe.layer_norm(x.half(), None, None, None, 1e-5, None, x, None, None)
    with pytest.raises(ValueError, match=r"x: expected \[rows, d\]"):
        moe.layer_norm(x[0], None, None, None, 1e-5, None, x, None, None)

    class Cuda(torch.Tensor):
        is_cuda = True

        def get_device(self):
            return 0

    c = lambda t: torch.Tensor._make_subclass(Cuda, t)
    arg = moe.block._arg
    assert arg(None, torch.float32, "x", 4, 0) is None
    t = c(torch.zeros(4))
    assert arg(t, torch.float32, "x", 4, 0) == t.data_ptr()
    with pytest.raises(ValueError, match="x: 4 elements, 5 needed"):
        arg(t, torch.float32, "x", 5, 0)
    with pytest.raises(TypeError, match="x: expected torch.bfloat16"):
        arg(t, torch.bfloat16, "x", 4, 0)
    with pytest.raises(ValueError, match="current device is cuda:1"):
        arg(t, torch.float32, "x", 4, 1)
    with pytest.raises(ValueError, match="x: must be contiguous"):
        arg(c(torch.zeros(4, 4).t()), torch.float32, "x", 4, 0)
    with pytest.raises(TypeError, match="x: expected a torch.Tensor"):
        arg(4096, torch.float32, "x", 4, 0)


# ------------------------------------------- formulas against differences --

def _differences(f, x, step):
    """Central differences of the scalar f at every element of x."""
    g = torch.zeros_like(x)
    flat, gf = x.view(-1), g.view(-1)
    for i in range(flat.numel()):
        v = flat[i].item()
        flat[i] = v + step
        hi = f()
        flat[i] = v - step
        gf[i] = (hi - f()) / (2 * step)
        flat[i] = v
    return g


def test_norm_gradient_formula_against_differences():
    """Third derivatives of the norm are O(1) at rows of unit size, so central
    differences with step 1e-4 are good to about 1e-8 times the gradient's
    size (truncation) plus 1e-12 (rounding)."""
    g = torch.Generator().manual_seed(1)
    n = lambda *s: torch.randn(*s, generator=g, dtype=torch.float64)
    x, dy, gamma, beta, dres = n(3, 16), n(3, 16), 1 + 0.1 * n(16), n(16), n(3, 16)

    def f():
        y = ref.norm(x, gamma, beta, 1e-5)[0]
        return (y * dy).sum() + (x * dres).sum()

    _, mean, rstd = ref.norm(x, gamma, beta, 1e-5)
    dx, dgamma, dbeta = ref.norm_backward(x, dy, gamma, mean, rstd, dres)
    for got, at in ((dx, x), (dgamma, gamma), (dbeta, beta)):
        assert (got - _differences(f, at, 1e-4)).abs().max() < 1e-6 * (1 + got.abs().max())


def test_balance_gradient_formula_against_differences():
    g = torch.Generator().manual_seed(2)
    T, N, K = 9, 6, 2
    logits = torch.randn(T, N, generator=g, dtype=torch.float64)
    idx = torch.topk(logits, K, 1).indices
    mask = torch.tensor([1, 1, 0, 1, 1, 1, 0, 1, 1])
    dlosses = torch.tensor([0.7, 0.3], dtype=torch.float64)
    r = ref.balance(logits, idx, mask, N)
    # the counts are held fixed (they are piecewise constant)
    d = ref.balance_backward(logits, idx, mask, r["expert_count"], r["token_count"], dlosses, None)
    f = lambda: (ref.balance(logits, idx, mask, N)["losses"] * dlosses).sum()
    assert (d - _differences(f, logits, 1e-5)).abs().max() < 1e-8
    assert torch.all(d[mask == 0] == 0)
    # the gates' share is added at the chosen experts
    dlogit = torch.randn(T, K, generator=g, dtype=torch.float64)
    e = ref.balance_backward(logits, idx, mask, r["expert_count"], r["token_count"], dlosses, dlogit)
    assert torch.allclose(e - d, torch.zeros(T, N, dtype=torch.float64).scatter(1, idx, dlogit))


def test_mxint8_reference_on_worked_blocks():
    """Hand-worked blocks of the format's rules."""
    v = torch.zeros(32)
    v[0], v[1], v[2], v[3] = 1.0, 0.5, -0.0078125, 0.0234375  # E = 0, step 1/64
    q, s = ref.mxint8(v.bfloat16()[None])
    assert s.item() == 127
    assert q[0, :4].tolist() == [64, 32, 0, 2]           # -0.5 -> 0 and 1.5 -> 2: ties to even
    v = torch.zeros(32)
    v[0], v[1] = 1.9921875, -1.9921875                   # 127.5 steps: held to 127
    q, s = ref.mxint8(v.bfloat16()[None])
    assert s.item() == 127 and q[0, :2].tolist() == [127, -127]
    q, s = ref.mxint8(torch.zeros(1, 32).bfloat16())
    assert s.item() == 0 and not q.any()
    v = torch.zeros(32)
    v[5] = 2.0 ** -133                                   # the smallest bf16
    q, s = ref.mxint8(v.bfloat16()[None])
    assert s.item() == 0 and q[0, 5].item() == 1
    assert ref.mxint8_value(q, s)[0, 5].item() == 2.0 ** -133
    v = torch.full((32,), 3.3895313892515355e38)         # the largest bf16
    q, s = ref.mxint8(v.bfloat16()[None])
    assert s.item() == 254 and q[0, 0].item() == 127
    for bad in (float("nan"), float("inf"), -float("inf")):
        v = torch.ones(32)
        v[31] = bad
        q, s = ref.mxint8(v.bfloat16()[None])
        assert s.item() == 255 and not q.any()
        assert torch.isnan(ref.mxint8_value(q, s)).all()


def test_mxint8_error_bound():
    """|value - v| <= half a step, 2^(E-7), or one step at the held top."""
    g = torch.Generator().manual_seed(3)
    v = (torch.randn(64, 256, generator=g) * torch.exp(3 * torch.randn(64, 1, generator=g))).bfloat16()
    q, s = ref.mxint8(v)
    step = torch.exp2(s.double() - 133).repeat_interleave(32, 1)
    err = (ref.mxint8_value(q, s) - v.double()).abs()
    assert torch.all(err <= step * torch.where(q.abs() == 127, 1.0, 0.5))


def test_local_arrays_read_as_pairs_are_aligned_for_them():
    """A float array of a kernel that is read as float2 has float2's alignment:
    without it the access is misaligned if the array ever lands in memory."""
    import os
    import re
    src = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                       "combine_expert_gemm_gb300", "csrc", "balance.cu")
    text = open(src).read()
    names = set(re.findall(r"reinterpret_cast<float2 \*>\((\w+)\)", text)) - {"p"}   # p: global rows
    assert names == {"acc", "v", "f"}
    for n in names:
        decl = re.findall(r"^ *(.*float %s\[VPT\];)" % n, text, re.M)
        assert decl and all(d.startswith("alignas(float2)") for d in decl), n
