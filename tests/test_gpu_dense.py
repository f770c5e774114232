"""The dense operators (include/moe_dense.h) on the GPU against their definitions
in 64 bits.

Tolerances.  H = 2^-8 is bf16's half step (eps / 2), C = 2^-23: the tensor core cuts
an fp32 sum by at most 2^-23 of its size at each addition, and fp32 arithmetic
rounds by half of that.  The feed-forward bounds carry each stored rounding and
each sum of n terms (n C sum |terms|) through the formulas, element by element; the
products of two error terms, below 2^-8 of the bounds, are covered by 1% on
top.  The activations' slopes and second derivatives are below 1.13, and the
exponential adds at most 2^-20 relative.  Independent roundings rarely line up, so
the 2-norm is held closer: a rounding is at most H / sqrt(3) in the root mean
square, and at most six follow each other (H, the factor, the scale, dG, the sum,
the output): 6e-3.

Newton-Schulz: a step changes an error E of X by at most L |E|_F, L the largest
slope of the step's odd polynomial on the interval of the singular values (3.89 for
the default up to 1.21: 4 is used), and adds the rounding of its own.  A piece pair
is off by 2^-22; the five products with it that enter a step (S twice, S S, C's
two terms) come with weights a + 3 |b| r^2 + 5 |c| r^4 <= 42 on the default's
interval: delta = 64 2^-22 |X_k|_F covers them and the sums (groups of 48
additions, each cut by 2^-23 at most: 3 2^-18 would line up only if all terms had one
sign; the random ones stay below 2^-19).  The result is off by at most
sum_k 4^(steps - 1 - k) delta_k in the Frobenius norm."""
import pytest
import torch

import _dense_ref as ref
from _gpu_util import DEV

pytestmark = pytest.mark.gpu
BF, FP, D = torch.bfloat16, torch.float32, torch.float64
H, C = 2.0 ** -8, 2.0 ** -23


@pytest.fixture(scope="module")
def moe():
    import __graft_entry__
    __graft_entry__.build()
    import combine_expert_gemm_gb300 as m
    return m


def _ws(n):
    return torch.zeros(n, dtype=torch.uint8, device=DEV)


def _within(got, want, bound, what, norm=None):
    got = got.to(D).cpu()
    assert got.shape == want.shape, what
    err = (got - want).abs()
    bad = ~(err <= 1.01 * bound + 1e-30)
    assert not bad.any(), (f"{what}: {int(bad.sum())} of {bad.numel()} outside; "
                           f"worst {float((err / (bound + 1e-30)).max()):.3g} of the bound")
    if norm is not None and float(want.norm()) > 0:
        assert float(err.norm()) <= norm * float(want.norm()), f"{what}: {float(err.norm() / want.norm()):.3g}"


def _ffn_inputs(T, d, h, add, scale, seed=0):
    g = torch.Generator().manual_seed(seed * 1000003 + T * 8191 + d * 127 + h)
    r = lambda *s, std=1.0: (torch.randn(*s, generator=g) * std).to(BF)
    t = dict(x=r(T, d), wg=r(h, d, std=d ** -0.5), wu=r(h, d, std=d ** -0.5), wd=r(d, h, std=h ** -0.5),
             add=r(T, d) if add else None, scale=torch.rand(T, generator=g) if scale else None, dy=r(T, d),
             dx_in=r(T, d))
    if scale and T > 2:
        t["scale"][1] = 0.0  # a token that the shared expert leaves out
    return t


def _dev(t):
    return None if t is None else t.to(DEV)


def _forward(moe, t, act, save=True, ws=None):
    (T, d), h = t["x"].shape, t["wg"].shape[0]
    e = lambda *s: torch.full(s, float("nan"), dtype=BF, device=DEV)
    o = dict(y=e(T, d), h=e(T, h), p=e(T, h) if save else None, q=e(T, h) if save else None)
    ws = _ws(moe.gated_ffn_workspace_bytes(T, d, h)) if ws is None else ws
    ws[256:] = 0xFF  # NaNs: nothing of the workspace is read before it is written
    moe.gated_ffn(_dev(t["x"]), _dev(t["wg"]), _dev(t["wu"]), _dev(t["wd"]), _dev(t["add"]), _dev(t["scale"]),
                  o["y"], o["h"], o["p"], o["q"], ws, act=act)
    assert moe.read_device_error(ws) == 0
    return o


def _backward(moe, t, o, xt=BF, wt=FP):
    (T, d), h = t["x"].shape, t["wg"].shape[0]
    e = lambda dt, *s: torch.full(s, float("nan"), dtype=dt, device=DEV)
    g = dict(dx=e(xt, T, d), dw_gate=e(wt, h, d), dw_up=e(wt, h, d), dw_down=e(wt, d, h),
             dscale=e(wt, T) if t["scale"] is not None else None)
    ws = _ws(moe.gated_ffn_backward_workspace_bytes(T, d, h))
    ws[256:] = 0xFF
    moe.gated_ffn_backward(_dev(t["x"]), _dev(t["wg"]), _dev(t["wu"]), _dev(t["wd"]), _dev(t["scale"]), o["h"], o["p"],
                           o["q"], _dev(t["dy"]), _dev(t["dx_in"]), g["dx"], g["dw_gate"], g["dw_up"], g["dw_down"],
                           g["dscale"], ws)
    assert moe.read_device_error(ws) == 0
    return g


def _bounds(t, f, b=None, dt=BF):
    """The bounds of the docstring."""
    a = {k: t[k].to(D).abs() for k in ("x", "wg", "wu", "wd", "dy")}
    (T, d), h = a["x"].shape, a["wg"].shape[0]
    s = f["s"].abs()
    eg, eu = d * C * (a["x"] @ a["wg"].t()), d * C * (a["x"] @ a["wu"].t())
    eh = 1.13 * eg * f["u"].abs() + f["p"].abs() * eu + f["h"].abs() * 2.0 ** -20
    out = dict(h=eh + H * f["h"].abs())
    ep = 1.13 * eg + f["p"].abs() * 2.0 ** -20 + H * f["p"].abs()
    eq = 1.13 * (eg * f["u"].abs() + eu) + f["u"].abs() * 2.0 ** -19 + H * f["q"].abs()
    out.update(p=ep, q=eq, y=s * (out["h"] @ a["wd"].t() + h * C * (f["h"].abs() @ a["wd"].t())) + H * f["y"].abs())
    if b is None:
        return out
    o = H if dt is BF else C
    er = d * C * (a["dy"] @ a["wd"])
    edu = s * (b["r"].abs() * ep + f["p"].abs() * er) + H * b["du"].abs()
    edg = s * (b["r"].abs() * eq + f["q"].abs() * er) + H * b["dg"].abs()
    adu, adg = b["du"].abs(), b["dg"].abs()
    out["dx"] = (edg + 2 * h * C * adg) @ a["wg"] + (edu + 2 * h * C * adu) @ a["wu"] + o * b["dx"].abs()
    out["dw_gate"] = (edg + T * C * adg).t() @ a["x"] + o * b["dw_gate"].abs()
    out["dw_up"] = (edu + T * C * adu).t() @ a["x"] + o * b["dw_up"].abs()
    es = s * out["h"] + (H * s * f["h"].abs() if t["scale"] is not None else 0.0)
    out["dw_down"] = a["dy"].t() @ (es + T * C * s * f["h"].abs()) + o * b["dw_down"].abs()
    out["dscale"] = ((b["r"].abs() * out["h"] + er * f["h"].abs() + h * C * (b["r"] * f["h"]).abs()).sum(1) +
                     o * b["dscale"].abs())
    return out


FFN = [(1, 8, 8), (1, 64, 128), (2, 72, 40), (7, 200, 136), (31, 64, 64), (33, 136, 264), (64, 512, 256), (65, 520, 72),
       (127, 128, 384), (129, 256, 128), (255, 264, 520), (257, 520, 264), (300, 1000, 712), (700, 256, 1416),
       (1100, 64, 2056), (1100, 2056, 64), (2500, 1000, 1416)]


@pytest.mark.parametrize("T,d,h", FFN)
@pytest.mark.parametrize("act,add,scale", [("silu", False, False), ("gelu", True, True), ("relu", True, False)])
def test_gated_ffn_forward(moe, T, d, h, act, add, scale):
    t = _ffn_inputs(T, d, h, add, scale)
    f = ref.ffn(t["x"], t["wg"], t["wu"], t["wd"], t["add"], t["scale"], act)
    b = _bounds(t, f)
    o = _forward(moe, t, act)
    for k in ("h", "y"):
        _within(o[k], f[k], b[k], k, 6e-3)
    if act != "relu":  # relu's slope jumps at 0, where G's last bits decide
        for k in ("p", "q"):
            _within(o[k], f[k], b[k], k, 6e-3)
    # without saving: the same bits
    n = _forward(moe, t, act, save=False)
    assert torch.equal(n["y"], o["y"]) and torch.equal(n["h"], o["h"])


@pytest.mark.parametrize("T,d,h", FFN)
@pytest.mark.parametrize("act,scale,xt,wt", [("silu", False, BF, FP), ("gelu", True, FP, BF), ("silu", True, BF, BF)])
def test_gated_ffn_backward(moe, T, d, h, act, scale, xt, wt):
    t = _ffn_inputs(T, d, h, True, scale, seed=1)
    t["dx_in"] = t["dx_in"].to(xt) if scale else None
    f = ref.ffn(t["x"], t["wg"], t["wu"], t["wd"], t["add"], t["scale"], act)
    b = ref.ffn_backward(f, t["x"], t["wg"], t["wu"], t["wd"], t["dy"], t["dx_in"])
    o = _forward(moe, t, act)
    g = _backward(moe, t, o, xt, wt)
    e = _bounds(t, f, b, wt)
    _within(g["dx"], b["dx"], _bounds(t, f, b, xt)["dx"], "dx", 6e-3)
    for k in ("dw_gate", "dw_up", "dw_down"):
        _within(g[k], b[k], e[k], k, 6e-3)
    if scale:
        _within(g["dscale"], b["dscale"], e["dscale"], "dscale")


def test_gated_ffn_no_tokens(moe):
    t = _ffn_inputs(0, 64, 128, True, True)
    o = _forward(moe, t, "silu")
    g = _backward(moe, t, o)
    for k in ("dw_gate", "dw_up", "dw_down"):
        assert not g[k].any()


@pytest.mark.parametrize("T,d,h", [(5, 64, 72), (300, 264, 128), (9000, 520, 264)])
def test_gated_ffn_in_place_and_rows_behind(moe, T, d, h):
    t = _ffn_inputs(T, d, h, True, True, seed=2)
    o = _forward(moe, t, "silu")
    g = _backward(moe, t, o)
    # y over add, dx over dx_in, buffers that go on behind the last row
    pad = lambda v: torch.cat([v, torch.full((40, v.shape[1]), 7.0, dtype=v.dtype)]).to(DEV)
    y, dx = pad(t["add"]), pad(t["dx_in"])
    hb, pb, qb = (pad(torch.zeros(T, h, dtype=BF)) for _ in range(3))
    ws = _ws(max(moe.gated_ffn_workspace_bytes(T, d, h), moe.gated_ffn_backward_workspace_bytes(T, d, h)))
    w = [_dev(t[k]) for k in ("x", "wg", "wu", "wd")]
    moe.gated_ffn(*w, y, _dev(t["scale"]), y, hb, pb, qb, ws)
    dw = [torch.empty(s, device=DEV) for s in ((h, d), (h, d), (d, h))]
    moe.gated_ffn_backward(*w, _dev(t["scale"]), hb, pb, qb, _dev(t["dy"]), dx, dx, *dw, None, ws)
    for buf, want in ((y, o["y"]), (hb, o["h"]), (pb, o["p"]), (qb, o["q"]), (dx, g["dx"])):
        assert torch.equal(buf[:T], want)
        assert bool((buf[T:] == 7.0).all())
    for a, k in zip(dw, ("dw_gate", "dw_up", "dw_down")):
        assert torch.equal(a, g[k])


@pytest.mark.parametrize("T", [12, 140, 1200])
def test_gated_ffn_non_finite_rows_stay_their_own(moe, T):
    t = _ffn_inputs(T, 136, 72, True, False, seed=3)
    clean = _forward(moe, t, "gelu")
    t["x"][3] = float("nan")
    t["x"][T - 1, 5] = float("inf")
    o = _forward(moe, t, "gelu")
    keep = [i for i in range(T) if i not in (3, T - 1)]
    assert torch.equal(o["y"][keep], clean["y"][keep])
    assert bool(o["y"][3].isnan().all()) and not bool(o["y"][T - 1].isfinite().all())


def test_gated_ffn_large_arguments(moe):
    # gates far out on both sides: the slope is 0 or 1 there, never a NaN
    T, d, h = 4, 8, 8
    t = _ffn_inputs(T, d, h, False, False)
    t["x"] = torch.eye(8)[:4].mul(1e4).to(BF)  # sums of one product: G and U are exact
    t["x"][1:2] *= -1
    t["x"][2:3] *= 1e16
    t["x"][3:4] *= -1e16
    t["wg"] = torch.ones(h, d).to(BF)
    t["wu"] = torch.ones(h, d).mul(1e-4).to(BF)
    for act in ("silu", "gelu", "relu"):
        o = _forward(moe, t, act)
        f = ref.ffn(t["x"], t["wg"], t["wu"], t["wd"], None, None, act)
        for k in ("p", "q", "h"):
            assert bool(o[k].isfinite().all()), (act, k)
            _within(o[k], f[k], H * f[k].abs() * 1.01, f"{act} {k}")


@pytest.mark.parametrize("T", [3, 200, 20000])
def test_gated_ffn_streams_graphs_and_repeats(moe, T):
    d, h = 256, 128
    t = _ffn_inputs(T, d, h, True, True, seed=4)
    o = _forward(moe, t, "silu")
    g = _backward(moe, t, o)
    w = [_dev(t[k]) for k in ("x", "wg", "wu", "wd")]
    sc, add, dy, dx_in = (_dev(t[k]) for k in ("scale", "add", "dy", "dx_in"))
    e = lambda *s: torch.empty(*s, dtype=BF, device=DEV)

    class Run:
        def __init__(self):
            self.ws = _ws(max(moe.gated_ffn_workspace_bytes(T, d, h), moe.gated_ffn_backward_workspace_bytes(T, d, h)))
            self.y, self.dx = e(T, d), e(T, d)
            self.hpq = [e(T, h) for _ in range(3)]
            self.dw = [torch.empty(s, device=DEV) for s in ((h, d), (h, d), (d, h))]

        def __call__(self, stream=None):
            moe.gated_ffn(*w, add, sc, self.y, *self.hpq, self.ws, stream=stream)
            moe.gated_ffn_backward(*w, sc, *self.hpq, dy, dx_in, self.dx, *self.dw, None, self.ws, stream=stream)

        def check(self):
            assert torch.equal(self.y, o["y"]) and torch.equal(self.dx, g["dx"])
            for a, k in zip(self.dw, ("dw_gate", "dw_up", "dw_down")):
                assert torch.equal(a, g[k])

    runs = [Run(), Run()]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in runs]
    for _ in range(3):
        for r, s in zip(runs, streams):  # two at once, each with its workspace
            r(stream=s)
    torch.cuda.synchronize()
    for r in runs:
        r.check()
    graph = torch.cuda.CUDAGraph()
    run = Run()
    run()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        run()
    for b in [run.y, run.dx] + run.hpq + run.dw:
        b.zero_()
    graph.replay()
    graph.replay()
    torch.cuda.synchronize()
    run.check()


def test_gated_ffn_argument_checks(moe):
    t = {k: _dev(v) for k, v in _ffn_inputs(4, 64, 128, True, True).items()}
    ws = _ws(moe.gated_ffn_workspace_bytes(4, 64, 128))
    y, h = torch.empty(4, 64, dtype=BF, device=DEV), torch.empty(4, 128, dtype=BF, device=DEV)
    ok = [t["x"], t["wg"], t["wu"], t["wd"], t["add"], t["scale"], y, h, None, None, ws]
    moe.gated_ffn(*ok)
    for i, bad, err in [(0, t["x"].float(), TypeError), (0, t["x"].cpu(), ValueError), (0, t["x"][0], ValueError),
                        (1, t["wg"].t(), ValueError), (1, t["wg"][:, :32], ValueError), (2, t["wu"][:64], ValueError),
                        (4, t["add"][:2], ValueError), (5, t["scale"].to(BF), TypeError), (6, y[:3], ValueError),
                        (7, h[:3], ValueError), (8, h, moe.MoEError), (10, ws[:16], moe.MoEError)]:
        args = list(ok)
        args[i] = bad
        with pytest.raises(err):
            moe.gated_ffn(*args)
    with pytest.raises(ValueError):
        moe.gated_ffn(*ok, act="tanh")


def test_gated_ffn_past_32_bit_offsets(moe):
    # x, y, dy and dx have more than 2^31 elements; the last rows are checked
    T, d, h, n = 1050001, 2056, 8, 50
    g = torch.Generator(device=DEV).manual_seed(1)
    r = lambda *s, std=1.0: (torch.randn(*s, generator=g, device=DEV, dtype=BF) * std)
    x, dy = r(T, d), r(T, d)
    wg, wu, wd = r(h, d, std=d ** -0.5), r(h, d, std=d ** -0.5), r(d, h, std=h ** -0.5)
    y, dx = torch.empty_like(x), torch.empty_like(x)
    hb, p, q = (torch.empty(T, h, dtype=BF, device=DEV) for _ in range(3))
    ws = _ws(max(moe.gated_ffn_workspace_bytes(T, d, h), moe.gated_ffn_backward_workspace_bytes(T, d, h)))
    dw = [torch.empty(s, device=DEV) for s in ((h, d), (h, d), (d, h))]
    moe.gated_ffn(x, wg, wu, wd, None, None, y, hb, p, q, ws)
    moe.gated_ffn_backward(x, wg, wu, wd, None, hb, p, q, dy, None, dx, *dw, None, ws)
    assert moe.read_device_error(ws) == 0
    t = dict(x=x[-n:].cpu(), wg=wg.cpu(), wu=wu.cpu(), wd=wd.cpu(), add=None, scale=None, dy=dy[-n:].cpu())
    f = ref.ffn(t["x"], t["wg"], t["wu"], t["wd"], None, None, "silu")
    b = ref.ffn_backward(f, t["x"], t["wg"], t["wu"], t["wd"], t["dy"], None)
    e = _bounds(t, f, b)
    _within(y[-n:], f["y"], e["y"], "y", 6e-3)
    _within(dx[-n:], b["dx"], e["dx"], "dx", 6e-3)


@pytest.mark.parametrize("T", [1, 20, 60, 100])
def test_gated_ffn_reads_weights_written_just_before(moe, T):
    """The second product's weights are loaded while the first runs: they are those that
    the kernel ahead of the call has written."""
    d, h = 1024, 512
    t = _ffn_inputs(T, d, h, False, False, seed=5)
    x, wg, wu, wd = (_dev(t[k]) for k in ("x", "wg", "wu", "wd"))
    sources = [(wd * s).contiguous() for s in (1.0, -2.0, 0.5)]
    y, hb = torch.empty(T, d, dtype=BF, device=DEV), torch.empty(T, h, dtype=BF, device=DEV)
    ws = _ws(moe.gated_ffn_workspace_bytes(T, d, h))
    want = []
    for s in sources:
        moe.gated_ffn(x, wg, wu, s, None, None, y, hb, None, None, ws)
        torch.cuda.synchronize()
        want.append(y.clone())
    live, got = torch.empty_like(wd), []
    for i in range(30):
        live.copy_(sources[i % 3])
        moe.gated_ffn(x, wg, wu, live, None, None, y, hb, None, None, ws)
        got.append(y.clone())
    for i, g in enumerate(got):
        assert torch.equal(g, want[i % 3]), i


# ------------------------------------------------------------ Newton-Schulz --

def _mats(B, rows, cols, seed=0, floor=0.3):
    g = torch.Generator().manual_seed(seed * 7907 + B * 31 + rows * 5 + cols)
    r = max(1, min(rows, cols) // 8)
    m = torch.randn(B, rows, r, generator=g) * torch.exp(-3.0 * torch.arange(r) / r) @ torch.randn(B, r, cols, generator=g)
    return 1e-3 * (m * r ** -0.5 + floor * torch.randn(B, rows, cols, generator=g))


def _ns_bound(norms, steps, L=4.0):
    return sum(L ** (steps - 1 - k) * 64 * 2.0 ** -22 * norms[k] for k in range(steps))


def _ns(moe, m, out=None, dt=FP, **kw):
    B, rows, cols = m.shape
    out = torch.full((B, rows, cols), float("nan"), dtype=dt, device=DEV) if out is None else out
    ws = _ws(moe.newton_schulz_workspace_bytes(B, rows, cols))
    ws[256:] = 0xFF  # NaNs: nothing of the workspace is read before it is written
    moe.newton_schulz(m if m.is_cuda else m.to(DEV), out, ws, **kw)
    assert moe.read_device_error(ws) == 0
    return out


def _check_ns(got, want, bound, what):
    err = (got.to(D).cpu() - want).square().sum((1, 2)).sqrt()
    half = torch.finfo(got.dtype).eps / 2 * want.square().sum((1, 2)).sqrt()
    assert bool((err <= bound + half).all()), f"{what}: {float((err / (bound + half)).max()):.3g} of the bound"


SIZES = [(1, 1, 1), (2, 1, 9), (1, 9, 1), (3, 7, 5), (2, 16, 64), (5, 33, 31), (2, 64, 64), (1, 130, 70), (3, 100, 300),
         (2, 255, 257), (1, 257, 256), (2, 256, 128), (1, 513, 700), (9, 128, 256), (40, 60, 128), (1, 1000, 90),
         # more tiles than SMs
         (40, 130, 300), (160, 60, 128), (200, 33, 20), (2, 1100, 1201), (30, 300, 200), (2, 1303, 1000)]


@pytest.mark.parametrize("B,rows,cols", SIZES)
def test_newton_schulz(moe, B, rows, cols):
    m = _mats(B, rows, cols)
    want, norms = ref.newton_schulz(m)
    got = _ns(moe, m)
    _check_ns(got, want, _ns_bound(norms, 5), "fp32")
    # a bf16 output is the fp32 one, rounded
    assert torch.equal(_ns(moe, m, dt=BF), got.to(BF))
    mb = m.to(BF)
    want, norms = ref.newton_schulz(mb)
    _check_ns(_ns(moe, mb, dt=BF), want, _ns_bound(norms, 5), "bf16")


def test_newton_schulz_transposes(moe):
    m = _mats(2, 90, 200)
    a, b = _ns(moe, m), _ns(moe, m.transpose(1, 2).contiguous())
    want, norms = ref.newton_schulz(m)
    _check_ns(b.transpose(1, 2).contiguous(), want, _ns_bound(norms, 5), "transposed")
    _check_ns(a, want, _ns_bound(norms, 5), "straight")


@pytest.mark.parametrize("B,rows,cols", [(2, 60, 77), (1, 150, 300), (40, 301, 130), (40, 130, 301)])
def test_newton_schulz_coefficients_in_place_and_unaligned(moe, B, rows, cols):
    m = _mats(B, rows, cols)
    cubic = (1.5, -0.5, 0.0)
    # c = 0 and a c that is small beside b among them
    coef = [ref.COEF, ref.COEF, (2.0, -1.5, 0.5), cubic, (1.5, -0.5, 1e-3), cubic, cubic]
    want, norms = ref.newton_schulz(m, 7, coef)
    # the slopes of the third step and of the cubics are below the default's
    _check_ns(_ns(moe, m, steps=7, coefficients=coef), want, _ns_bound(norms, 7), "per step")
    want, norms = ref.newton_schulz(m, 4, [cubic] * 4)
    _check_ns(_ns(moe, m, steps=4, coefficients=cubic), want, _ns_bound(norms, 4), "one triple")
    want, norms = ref.newton_schulz(m, 1)
    _check_ns(_ns(moe, m, steps=1), want, _ns_bound(norms, 1), "one step")
    for c in (torch.tensor(ref.COEF), torch.tensor([ref.COEF]), [list(ref.COEF)]):
        assert torch.equal(_ns(moe, m, steps=1, coefficients=c), _ns(moe, m, steps=1))
    # a shift of the square beyond its range: S is read instead (slopes below 4, and the
    # weights of the bound's rounding, a + 3 |b| r^2 + 5 |c| r^4, below 42)
    wide = [(3.0, -1.5, 0.05)] + [cubic] * 3
    want, norms = ref.newton_schulz(m, 4, wide)
    _check_ns(_ns(moe, m, steps=4, coefficients=wide), want, _ns_bound(norms, 4), "wide shift")
    plain = _ns(moe, m)
    buf = torch.zeros(m.numel() + 1, device=DEV)
    view = buf[1:].view(B, rows, cols)  # 4-byte aligned only
    view.copy_(m)
    _ns(moe, view, out=view)
    assert torch.equal(view, plain) and float(buf[0]) == 0.0


@pytest.mark.parametrize("rows,cols", [(40, 50), (140, 300), (900, 1000)])
def test_newton_schulz_special_matrices(moe, rows, cols):
    m = _mats(4, rows, cols)
    clean = _ns(moe, m)
    m[1] = 0.0
    m[2, 3, 4] = float("nan")
    m[3, 0, 0] = float("inf")
    got = _ns(moe, m)
    assert torch.equal(got[0], clean[0]) and not bool(got[1].any())
    assert bool(got[2].isnan().all()) and bool(got[3].isnan().all())
    # tiny and huge scales give the same factor, as long as eps is small beside them
    for scale in (1e-8, 1e12):
        s = _ns(moe, m[:1] * scale, eps=1e-20)
        want, norms = ref.newton_schulz(m[:1] * scale, eps=1e-20)
        _check_ns(s, want, _ns_bound(norms, 5), f"scale {scale}")
    # orthogonal rows already: singular values all alike
    q = torch.linalg.qr(torch.randn(rows, rows, generator=torch.Generator().manual_seed(1)))[0].contiguous()[None]
    want, norms = ref.newton_schulz(q)
    _check_ns(_ns(moe, q), want, _ns_bound(norms, 5), "orthogonal")
    # one direction only
    one = torch.outer(torch.arange(1.0, rows + 1), torch.arange(1.0, cols + 1))[None]
    want, norms = ref.newton_schulz(one)
    _check_ns(_ns(moe, one), want, _ns_bound(norms, 5), "rank one")


@pytest.mark.parametrize("B,rows,cols,nesterov,copy", [(2, 60, 40, True, True), (1, 128, 300, False, True),
                                                      (3, 33, 65, True, False), (8, 256, 128, True, True),
                                                      (1, 300, 200, True, True), (40, 131, 300, True, True),
                                                      (40, 300, 131, True, True), (40, 300, 136, False, False)])
def test_muon_step(moe, B, rows, cols, nesterov, copy):
    g = torch.Generator().manual_seed(rows)
    w = torch.randn(B, rows, cols, generator=g) * cols ** -0.5
    v = _mats(B, rows, cols, 5)
    lr, mu, wd, scale = 0.03, 0.9, 0.2, 1.7
    wt, vt, lrt = w.to(DEV), v.to(DEV), torch.tensor([lr], device=DEV)
    wc = torch.empty(B, rows, cols, dtype=BF, device=DEV) if copy else None
    ws = _ws(moe.newton_schulz_workspace_bytes(B, rows, cols))
    lr32, mu32, wd32, scale32 = (float(torch.tensor(q)) for q in (lr, mu, wd, scale))
    for step in range(3):
        grad = _mats(B, rows, cols, 10 + step)
        w0, v0 = wt.cpu(), vt.cpu()
        moe.muon_step(wt, wc, vt, grad.to(DEV), lrt, mu, wd, scale, ws, nesterov=nesterov)
        # the step's own formula from the state that it found
        vn = v0.to(D) * mu32 + grad.to(D)
        assert bool(((vt.cpu().to(D) - vn).abs() <= 2.0 ** -24 * vn.abs() + 1e-45).all())
        u = grad.to(D) + mu32 * vt.cpu().to(D) if nesterov else vt.cpu().to(D)
        o, norms = ref.newton_schulz(u)
        want = (1 - lr32 * wd32) * w0.to(D) - lr32 * scale32 * o
        err = (wt.cpu().to(D) - want).square().sum((1, 2)).sqrt()
        # the factor's bound, and roundings of lr wd, lr scale, their products and the sum
        bound = lr32 * scale32 * (_ns_bound(norms, 5) + 3 * 2.0 ** -24 * o.norm()) + 4 * 2.0 ** -24 * w0.to(D).norm()
        assert bool((err <= bound).all()), float((err / bound).max())
        if copy:
            assert torch.equal(wc, wt.to(BF))
    assert moe.read_device_error(ws) == 0


@pytest.mark.parametrize("B,rows,cols", [(2, 96, 64), (1, 160, 300), (40, 160, 300)])
def test_muon_step_captured(moe, B, rows, cols):
    w = torch.randn(B, rows, cols, generator=torch.Generator().manual_seed(2)).to(DEV)
    v, grad = torch.zeros(B, rows, cols, device=DEV), _mats(B, rows, cols).to(DEV)
    lr = torch.tensor([0.1], device=DEV)
    ws = _ws(moe.newton_schulz_workspace_bytes(B, rows, cols))
    args = (None, v, grad, lr, 0.9, 0.0, 1.0, ws)
    start = w.clone()
    moe.muon_step(w, *args)
    moe.muon_step(w, *args)
    lr.fill_(0.01)
    moe.muon_step(w, *args)
    want, want_v = w.clone(), v.clone()
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        moe.muon_step(w, *args)
    w.copy_(start)
    v.zero_()
    lr.fill_(0.1)
    graph.replay()
    graph.replay()
    lr.fill_(0.01)  # a schedule between replays
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(w, want) and torch.equal(v, want_v)


def test_muon_past_32_bit_offsets(moe):
    # more than 2^31 elements; the last matrix against the same step of it alone
    B, rows, cols = 130, 4096, 4100
    g = torch.Generator(device=DEV).manual_seed(2)
    w = torch.randn(B, rows, cols, generator=g, device=DEV)
    grad = torch.randn(B, rows, cols, generator=g, device=DEV)
    v = torch.zeros_like(w)
    lr = torch.tensor([0.1], device=DEV)
    last = [t[-1:].clone() for t in (w, v, grad)]
    ws = _ws(moe.newton_schulz_workspace_bytes(B, rows, cols))
    moe.muon_step(w, None, v, grad, lr, 0.9, 0.0, 1.0, ws, steps=2)
    assert moe.read_device_error(ws) == 0
    moe.muon_step(last[0], None, last[1], last[2], lr, 0.9, 0.0, 1.0, ws, steps=2)
    assert torch.equal(v[-1:], last[1])
    # the norms are summed in another order: 2^-20 of the factor covers it; and two sums
    # on either side of a rounding boundary become neighbouring fp32 values, which are
    # 2^-23 of an element apart at most
    assert float((w[-1:] - last[0]).norm()) <= 2.0 ** -20 * 0.1 * 3.4445 ** 2 + 2.0 ** -23 * float(last[0].norm())


def test_newton_schulz_argument_checks(moe):
    m = _mats(2, 20, 30).to(DEV)
    ws = _ws(moe.newton_schulz_workspace_bytes(2, 20, 30))
    out = torch.empty_like(m)
    moe.newton_schulz(m, out, ws)
    moe.newton_schulz(m[0], out[0], ws)
    for a, err in [((m.half(), out, ws), TypeError), ((m[0, 0], out, ws), ValueError), ((m, out[:1], ws), ValueError),
                   ((m, out, ws[:200]), moe.MoEError), ((m.cpu(), out, ws), ValueError),
                   ((m.transpose(1, 2), out, ws), ValueError)]:
        with pytest.raises(err):
            moe.newton_schulz(*a)
    with pytest.raises(ValueError):
        moe.newton_schulz(m, out, ws, steps=3, coefficients=[(1, 0, 0)] * 2)
    with pytest.raises(moe.MoEError):
        moe.newton_schulz(m, out, ws, coefficients=(9.0, 0.0, 0.0))
    with pytest.raises(ValueError):
        moe.muon_step(m, None, out[:1], m, torch.zeros(1, device=DEV), 0.9, 0.0, 1.0, ws)
