"""The dense operators (include/moe_dense.h) on the CPU: refusals before anything
is enqueued, and the formulas that the GPU tests use compared with differences
and with a singular value decomposition."""
import ctypes
import math

import pytest
import torch

import _dense_ref as ref


@pytest.fixture(scope="module")
def moe():
    import __graft_entry__
    __graft_entry__.build()
    import combine_expert_gemm_gb300 as m
    return m


def P(i):
    return ctypes.c_void_p(4096 * (i + 1))


MIS = ctypes.c_void_p(4096 + 8)


def test_gated_ffn_refusals(moe):
    lib = moe.lib()
    need = lib.moe_gated_ffn_workspace_bytes(4, 64, 128)
    assert need >= 256
    for bad in ((-1, 64, 128), (4, 0, 128), (4, 64, -8), (4, 12, 128), (4, 64, 100), (4, 65544, 64),
                (4, 64, 65544), ((1 << 24) + 1, 64, 64)):
        assert lib.moe_gated_ffn_workspace_bytes(*bad) == 0, bad
        assert lib.moe_gated_ffn_backward_workspace_bytes(*bad) == 0, bad
    names = ["x", "w_gate", "w_up", "w_down", "add", "token_scale", "y", "h_act", "p_save", "q_save"]

    def call(T=4, d=64, h=128, act=0, ws=P(40), n=need, **kw):
        a = [kw.get(k, P(i)) for i, k in enumerate(names)]
        return lib.moe_gated_ffn(T, d, h, act, *a, ws, n, None)

    assert call(T=-1) == 1 and call(d=0) == 1 and call(d=60) == 2 and call(h=4) == 2
    assert call(d=1 << 20) == 5 and call(act=3) == 1 and call(act=-1) == 1
    for k in ("x", "w_gate", "w_up", "w_down", "y", "h_act", "p_save", "q_save"):
        assert call(**{k: None}) == 1, k              # p_save without q_save too
    for k in names:
        assert call(**{k: MIS}) == 2, k
    assert call(y=P(0)) == 1                          # y is x
    assert call(ws=None) == 3 and call(ws=MIS) == 3 and call(n=need - 1) == 3
    assert call(T=0, x=None, y=None, n=1 << 30) == 0  # nothing to do, nothing enqueued


def test_gated_ffn_backward_refusals(moe):
    lib = moe.lib()
    need = lib.moe_gated_ffn_backward_workspace_bytes(4, 64, 128)
    names = ["x", "w_gate", "w_up", "w_down", "token_scale", "h_act", "p_save", "q_save", "dy", "dx_in", "dx",
             "dw_gate", "dw_up", "dw_down", "dtoken_scale"]

    def call(T=4, d=64, h=128, xt=0, wt=1, ws=P(40), n=need, **kw):
        a = [kw.get(k, P(i)) for i, k in enumerate(names)]
        return lib.moe_gated_ffn_backward(T, d, h, *a[:9], xt, *a[9:11], wt, *a[11:], ws, n, None)

    assert call(T=-1) == 1 and call(d=60) == 2 and call(xt=2) == 1 and call(wt=-1) == 1
    for k in ("x", "w_gate", "w_up", "w_down", "h_act", "p_save", "q_save", "dy", "dx", "dw_gate", "dw_up", "dw_down"):
        assert call(**{k: None}) == 1, k
    assert call(token_scale=None) == 1                # dtoken_scale without token_scale
    for k in names:
        assert call(**{k: MIS}) == 2, k
    assert call(dx=P(0)) == 1 and call(dx=P(8)) == 1  # dx is x, dx is dy
    assert call(ws=None) == 3 and call(ws=MIS) == 3 and call(n=need - 1) == 3


def test_newton_schulz_refusals(moe):
    lib = moe.lib()
    need = lib.moe_newton_schulz_workspace_bytes(2, 30, 50)
    assert need > 0 and lib.moe_newton_schulz_workspace_bytes(0, 30, 50) >= 256
    for bad in ((-1, 30, 50), (2, 0, 50), (2, 30, -1), (2, 65537, 5), (65536, 30, 50), (60000, 65536, 65536)):
        assert lib.moe_newton_schulz_workspace_bytes(*bad) == 0, bad

    def call(B=2, rows=30, cols=50, xt=1, x=P(0), ot=0, out=P(1), steps=5, coef=None, eps=1e-7, ws=P(40), n=need):
        c = None if coef is None else (ctypes.c_float * len(coef))(*coef)
        return lib.moe_newton_schulz(B, rows, cols, xt, x, ot, out, steps, c, eps, ws, n, None)

    assert call(B=-1) == 1 and call(rows=0) == 1 and call(cols=65537) == 5
    assert call(xt=2) == 1 and call(ot=-1) == 1 and call(steps=0) == 1 and call(steps=17) == 1
    for eps in (0.0, -1.0, 1e-31, float("nan"), float("inf")):
        assert call(eps=eps) == 1
    assert call(x=None) == 1 and call(out=None) == 1
    assert call(out=P(0)) == 1                        # in place with two types
    assert call(x=ctypes.c_void_p(4098)) == 2 and call(out=ctypes.c_void_p(4097)) == 2
    assert call(ws=None) == 3 and call(ws=MIS) == 3 and call(n=need - 1) == 3
    assert call(steps=1, coef=[float("nan"), 0, 0]) == 1
    # singular values or the factor leave the pieces' range
    assert call(steps=1, coef=[8.0, 0, 0]) == 5 and call(steps=2, coef=[3.0, 0, 0] * 2) == 5
    assert call(steps=1, coef=[61.0, -120.0, 60.0]) == 5
    assert call(B=0, x=None, out=None) == 0


def test_muon_refusals(moe):
    lib = moe.lib()
    need = lib.moe_newton_schulz_workspace_bytes(2, 30, 50)
    names = ["w", "w_copy", "momentum", "grad", "lr"]

    def call(B=2, mu=0.9, wd=0.1, scale=1.0, steps=5, eps=1e-7, ws=P(40), n=need, **kw):
        a = [kw.get(k, P(i)) for i, k in enumerate(names)]
        return lib.moe_muon_step(B, 30, 50, *a, mu, wd, scale, 1, steps, None, eps, ws, n, None)

    for k in ("w", "momentum", "grad", "lr"):
        assert call(**{k: None}) == 1, k
        assert call(**{k: ctypes.c_void_p(4098)}) == 2, k
    assert call(w_copy=ctypes.c_void_p(4097)) == 2
    for a, b in (("w", 2), ("w", 3), ("w_copy", 0), ("w_copy", 2), ("momentum", 3), ("lr", 0)):
        assert call(**{a: P(b)}) == 1, (a, b)         # one buffer for two tensors
    for k in ("mu", "wd", "scale"):
        assert call(**{k: float("inf")}) == 1 and call(**{k: float("nan")}) == 1
    assert call(steps=0) == 1 and call(eps=0.0) == 1 and call(n=need - 1) == 3 and call(B=-1) == 1
    assert call(B=0, w=None) == 0


@pytest.mark.parametrize("name", ["silu", "gelu", "relu"])
def test_ffn_gradient_against_differences(name):
    g = torch.Generator().manual_seed(3)
    r = lambda *s: torch.randn(*s, generator=g, dtype=ref.D)
    x, wg, wu, wd, add, s, dy = r(5, 8), r(16, 8), r(16, 8), r(8, 16), r(5, 8), torch.rand(5, dtype=ref.D), r(5, 8)
    f = ref.ffn(x, wg, wu, wd, add, s, name)
    b = ref.ffn_backward(f, x, wg, wu, wd, dy, None)
    loss = lambda: float((ref.ffn(x, wg, wu, wd, add, s, name)["y"] * dy).sum())
    e = 1e-6
    for t, grad in ((x, b["dx"]), (wg, b["dw_gate"]), (wu, b["dw_up"]), (wd, b["dw_down"]), (s, b["dscale"])):
        flat, want = t.reshape(-1), grad.reshape(-1)
        for i in range(0, flat.numel(), max(1, flat.numel() // 7)):
            old = float(flat[i])
            flat[i] = old + e
            hi = loss()
            flat[i] = old - e
            lo = loss()
            flat[i] = old
            # rounding of the two losses over 2 e, and e^2 of the third derivative
            assert abs((hi - lo) / (2 * e) - float(want[i])) < 1e-5 * (1 + abs(float(want[i]))), name


@pytest.mark.parametrize("rows,cols", [(6, 9), (9, 6), (1, 4)])
def test_newton_schulz_acts_on_singular_values(rows, cols):
    g = torch.Generator().manual_seed(4)
    m = torch.randn(2, rows, cols, generator=g, dtype=ref.D)
    got, _ = ref.newton_schulz(m)
    u, s, v = torch.linalg.svd(m, full_matrices=False)
    s = s / (s.square().sum(1, keepdim=True).sqrt() + 1e-7)
    for _ in range(5):
        s = ref.COEF[0] * s + ref.COEF[1] * s ** 3 + ref.COEF[2] * s ** 5
    assert float((got - (u * s[:, None]) @ v).abs().max()) < 1e-9
    assert math.isclose(float(s.max()), 1.0, abs_tol=0.35)
