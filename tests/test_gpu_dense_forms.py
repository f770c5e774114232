"""The dense operators against 64 bits at sizes that reach each form of their products
(on a GPU of 152 SMs, which the forms' rules count), with the bounds of
test_gpu_dense.py.  A size's comment says which forms it adds."""
import pytest
import torch

import _dense_ref as ref
from _gpu_util import DEV
from test_gpu_dense import (BF, C, D, FP, H, _backward, _bounds, _check_ns, _ffn_inputs, _forward, _mats, _ns, _ns_bound,
                            _within, _ws)

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def moe():
    import __graft_entry__
    __graft_entry__.build()
    import combine_expert_gemm_gb300 as m
    return m


FFN_FORMS = [
    (20000, 72, 64),    # all products on pairs with narrow tiles
    (12000, 136, 136),  # wide tiles of all but the gradients; more than one tile a pair
    (700, 1416, 264),   # gradients in wide tiles, the weights' the longer
    (300, 2056, 264),   # the same, dx's the longer
    (2500, 1000, 1416), # several tiles a pair of one kind, shares evened out with the other
    (4100, 1416, 264),  # the other way round
    (9000, 520, 264),   # narrow gradients, more tokens than one accumulator's
]


@pytest.mark.parametrize("T,d,h", FFN_FORMS)
@pytest.mark.parametrize("act,scale,xt,wt", [("silu", True, BF, BF), ("gelu", True, FP, FP), ("relu", False, FP, BF),
                                             ("silu", False, BF, FP)])
def test_gated_ffn_forms(moe, T, d, h, act, scale, xt, wt):
    t = _ffn_inputs(T, d, h, True, scale, seed=8)
    t["dx_in"] = t["dx_in"].to(xt)
    f = ref.ffn(t["x"], t["wg"], t["wu"], t["wd"], t["add"], t["scale"], act)
    b = ref.ffn_backward(f, t["x"], t["wg"], t["wu"], t["wd"], t["dy"], t["dx_in"])
    o = _forward(moe, t, act)
    e = _bounds(t, f, b, wt)
    for k in ("h", "y"):
        _within(o[k], f[k], e[k], k, 6e-3)
    if act == "relu":
        return  # its slope jumps at 0, where G's last bits decide
    g = _backward(moe, t, o, xt, wt)
    _within(g["dx"], b["dx"], _bounds(t, f, b, xt)["dx"], "dx", 6e-3)
    for k in ("dw_gate", "dw_up", "dw_down"):
        _within(g[k], b[k], e[k], k, 6e-3)
    if scale:
        _within(g["dscale"], b["dscale"], e["dscale"], "dscale")


NS_FORMS = [
    (16, 130, 130),                                  # single SMs, 64 tokens a tile
    (30, 130, 133), (20, 200, 257),                  # symmetric products mirrored, without and with a split reduction
    (12, 300, 400), (12, 400, 300), (3, 1001, 717),  # the same with 128-token tiles in the other products
    (20, 70, 400), (16, 600, 90), (1, 301, 257),     # m of one tile; tall with 128 and 64 tokens
    (1, 1500, 1500),                                 # many tiles of one matrix
    (20, 257, 257), (4, 900, 1000), (4, 1000, 900),  # pairs, wide symmetric tiles, mirrored
    (40, 130, 257), (40, 257, 130),                  # narrow tiles of the last product, tall too
    (20, 400, 130), (6, 1100, 257),                  # narrow symmetric tiles, mirrored in the second
]


@pytest.mark.parametrize("B,rows,cols", NS_FORMS)
def test_newton_schulz_forms(moe, B, rows, cols):
    m = _mats(B, rows, cols, 3)
    want, norms = ref.newton_schulz(m)
    _check_ns(_ns(moe, m), want, _ns_bound(norms, 5), "fp32")
    _check_ns(_ns(moe, m, dt=BF), want, _ns_bound(norms, 5), "bf16")


CUBIC = (1.5, -0.5, 0.0)


@pytest.mark.parametrize("B,rows,cols", [(60, 40, 200), (16, 130, 130), (20, 200, 257), (12, 300, 400), (30, 130, 133),
                                         (20, 70, 400), (2, 1100, 1201), (4, 900, 1000), (40, 130, 257)])
def test_newton_schulz_forms_that_read_the_square(moe, B, rows, cols):
    """c small beside b, and a shift past its range: the second product reads S (slopes below
    4, weights of the bound's rounding below 42)."""
    m = _mats(B, rows, cols, 4)
    for coef in ([(1.5, -0.5, 1e-3)] + [CUBIC] * 2, [(3.0, -1.5, 0.05)] + [CUBIC] * 2):
        want, norms = ref.newton_schulz(m, 3, coef)
        _check_ns(_ns(moe, m, steps=3, coefficients=coef), want, _ns_bound(norms, 3), str(coef[0]))


@pytest.mark.parametrize("B,rows,cols,copy", [(12, 300, 400, True), (12, 400, 300, True), (20, 70, 401, True),
                                              (16, 600, 90, False), (4, 900, 1000, True), (4, 1000, 900, True),
                                              (40, 257, 130, True), (2, 1303, 1000, True), (3, 1001, 717, True)])
def test_muon_step_forms(moe, B, rows, cols, copy):
    g = torch.Generator().manual_seed(rows)
    w = torch.randn(B, rows, cols, generator=g) * cols ** -0.5
    v, grad = _mats(B, rows, cols, 5), _mats(B, rows, cols, 6)
    lr, mu, wd, scale = (float(torch.tensor(q)) for q in (0.03, 0.9, 0.2, 1.7))
    wt, vt = w.to(DEV), v.to(DEV)
    wc = torch.empty(B, rows, cols, dtype=BF, device=DEV) if copy else None
    ws = _ws(moe.newton_schulz_workspace_bytes(B, rows, cols))
    moe.muon_step(wt, wc, vt, grad.to(DEV), torch.tensor([lr], device=DEV), mu, wd, scale, ws)
    assert moe.read_device_error(ws) == 0
    vn = v.to(D) * mu + grad.to(D)
    assert bool(((vt.cpu().to(D) - vn).abs() <= 2.0 ** -24 * vn.abs() + 1e-45).all())
    o, norms = ref.newton_schulz(grad.to(D) + mu * vt.cpu().to(D))
    want = (1 - lr * wd) * w.to(D) - lr * scale * o
    err = (wt.cpu().to(D) - want).square().sum((1, 2)).sqrt()
    bound = lr * scale * (_ns_bound(norms, 5) + 3 * 2.0 ** -24 * o.norm()) + 4 * 2.0 ** -24 * w.to(D).norm()
    assert bool((err <= bound).all()), float((err / bound).max())
    if copy:
        assert torch.equal(wc, wt.to(BF))


@pytest.mark.parametrize("a,b", [((300, 40, 50), (300, 60, 30)), ((8, 128, 256), (12, 300, 400)),
                                 ((20, 70, 400), (4, 900, 1000)), ((3, 1001, 717), (2, 1303, 1000))])
def test_newton_schulz_on_two_streams(moe, a, b):
    """Two calls at once, each with its workspace, beside a few tokens' feed-forward on a
    third stream; and the same captured into one graph."""
    calls = []
    for s in (a, b):
        m = _mats(*s).to(DEV)
        calls.append((m, torch.empty_like(m), _ws(moe.newton_schulz_workspace_bytes(*s))))
    t = _ffn_inputs(20, 512, 256, True, True)
    w = [t[k].to(DEV) for k in ("x", "wg", "wu", "wd", "add", "scale")]
    y, hb = torch.empty(20, 512, dtype=BF, device=DEV), torch.empty(20, 256, dtype=BF, device=DEV)
    ws = _ws(moe.gated_ffn_workspace_bytes(20, 512, 256))

    def run(streams):
        for c, s in zip(calls, streams):
            moe.newton_schulz(*c, stream=s)
        moe.gated_ffn(*w, y, hb, None, None, ws, stream=streams[2])

    run([None] * 3)
    torch.cuda.synchronize()
    want = [c[1].clone() for c in calls] + [y.clone()]
    streams = [torch.cuda.Stream() for _ in range(3)]

    def check():
        torch.cuda.synchronize()
        for got, q in zip([c[1] for c in calls] + [y], want):
            assert torch.equal(got, q)
            got.zero_()
        torch.cuda.synchronize()
        assert all(moe.read_device_error(q) == 0 for q in (calls[0][2], calls[1][2], ws))

    for _ in range(3):
        for _ in range(4):
            run(streams)
        check()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        now = torch.cuda.current_stream()
        for s in streams:
            s.wait_stream(now)
        run(streams)
        for s in streams:
            now.wait_stream(s)
    for _ in range(2):
        graph.replay()
        check()
