"""The block operators (include/moe_block.h) on the GPU against their
definitions in 64 bits.

Tolerances.  u = 2^-24 is the unit roundoff of fp32.  A sum of n fp32 terms in
any order is within n u sum|terms| of the exact one; the kernels' sums are
trees whose depth is far below n, so n u is a safe bound and DEPTH = 128 covers
a row's sums (at most 64 terms a lane, 5 shuffles, 32 warps) and the handful of
roundings around them.  bf16 outputs add half an ulp, 2^-9 relative, written
as 2^-8 so that a result next to a rounding boundary may fall either way.
"""
import math

import numpy as np
import pytest
import torch

import _block_ref as ref
from _gpu_util import DEV

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
DEPTH = 128
BF, FP = torch.bfloat16, torch.float32
D = torch.float64


@pytest.fixture(scope="module")
def moe():
    import __graft_entry__
    __graft_entry__.build()
    import combine_expert_gemm_gb300 as m
    return m


def _gen(seed):
    return torch.Generator().manual_seed(seed)


def _within(got, want, bound, what):
    got, want = got.double().cpu(), want.double()
    assert got.shape == want.shape, what
    bad = ~((got - want).abs() <= bound)
    assert not bad.any(), (f"{what}: {int(bad.sum())} of {bad.numel()} outside; worst "
                           f"{((got - want).abs() / bound).nan_to_num(1e30).max():.3g} of the bound")


# -------------------------------------------------------------- layer norm --

def _run_norm(moe, x, add, gamma, beta, eps=1e-5, stats=True):
    T, d = x.shape
    x_sum = None if add is None else torch.empty_like(x)
    y = torch.empty(T, d, dtype=BF, device=DEV)
    mean, rstd = (torch.empty(T, device=DEV) for _ in range(2)) if stats else (None, None)
    moe.layer_norm(x, add, gamma, beta, eps, x_sum, y, mean, rstd)
    return x_sum, y, mean, rstd


def _run_norm_bwd(moe, x, dy, gamma, mean, rstd, dres, gt=BF, weights=True):
    T, d = x.shape
    dx = torch.empty(T, d, dtype=gt, device=DEV)
    dg, db = (torch.empty(d, device=DEV) for _ in range(2)) if weights else (None, None)
    ws = torch.zeros(moe.layer_norm_backward_workspace_bytes(T, d), dtype=torch.uint8, device=DEV)
    moe.layer_norm_backward(x, dy, gamma, mean, rstd, dres, dx, dg, db, ws)
    return dx, dg, db


def _norm_bounds(s, gamma, beta, eps):
    """(y, mean, rstd) in 64 bits with the fp32 error bounds of mean, rstd and xh."""
    y, mean, rstd = ref.norm(s, gamma, beta, eps)
    s = s.to(D)
    big = s.abs().amax(1)
    e_mean = DEPTH * U * s.abs().mean(1) + U * mean.abs()
    # rstd: relative error of the variance (its own sum, and the mean's error
    # against the deviation) halved, plus the square root and the division
    e_rstd = rstd * (DEPTH * U * (1 + big * rstd) ** 2 + 4 * U)
    xh = (s - mean[:, None]) * rstd[:, None]
    e_xh = (rstd * e_mean + 2 * U * big * rstd)[:, None] + xh.abs() * (e_rstd / rstd + 4 * U)[:, None]
    return y, mean, rstd, xh, e_mean, e_rstd, e_xh


@pytest.mark.parametrize("T,d,xt,yt,gt", [
    (1, 8, BF, FP, BF), (3, 64, FP, BF, FP), (37, 1000, FP, BF, BF), (300, 2048, BF, FP, BF),
    (65, 4096, BF, BF, FP), (7, 8200, FP, FP, FP), (5, 16384, BF, FP, BF), (1, 2048, BF, FP, BF),
    (1537, 136, BF, FP, BF), (2, 16376, FP, BF, BF), (513, 512, FP, FP, BF),
])
@pytest.mark.parametrize("kind", ["full", "bare"])
def test_layer_norm_and_backward(moe, T, d, xt, yt, gt, kind):
    g = _gen(T * 31 + d)
    n = lambda *s: torch.randn(*s, generator=g)
    full = kind == "full"
    x = (n(T, d) * (0.2 + 3 * torch.rand(T, 1, generator=g)) + 0.5).to(xt)
    add = n(T, d).to(BF) if full else None
    gamma, beta = (1 + 0.2 * n(d), 0.3 * n(d)) if full else (None, None)
    dy, dres = n(T, d).to(yt), n(T, d).to(gt) if full else None
    eps = 1e-5
    dev = lambda t: None if t is None else t.to(DEV)
    x_sum, y, mean, rstd = _run_norm(moe, dev(x), dev(add), dev(gamma), dev(beta), eps)
    s = x
    if full:
        s = (x.float() + add.float()).to(xt)
        assert torch.equal(x_sum.cpu(), s)                # one fp32 sum, rounded once
    wy, wm, wr, xh, e_mean, e_rstd, e_xh = _norm_bounds(s, gamma, beta, eps)
    ga = torch.ones(d, dtype=D) if gamma is None else gamma.to(D)
    _within(mean, wm, e_mean + 1e-30, "mean")
    _within(rstd, wr, e_rstd, "rstd")
    off = 0 if beta is None else beta.to(D).abs()
    _within(y, wy, 2.0 ** -8 * wy.abs() + e_xh * ga.abs() + 4 * U * off + 1e-30, "y")

    # the backward takes the forward's own mean and rstd as given
    dx, dg, db = _run_norm_bwd(moe, dev(s), dev(dy), dev(gamma), mean, rstd, dev(dres), gt)
    m, r = mean.cpu(), rstd.cpu()
    wdx, wdg, wdb = ref.norm_backward(s, dy, gamma, m, r, dres)
    sh = (s.to(D) - m.to(D)[:, None]) * r.to(D)[:, None]
    w = (dy.to(D) * ga).abs()
    e_s = 4 * U * (sh.abs() + (s.to(D).abs().amax(1) * r.to(D))[:, None])   # xh's own error
    mag = w + w.mean(1, keepdim=True) + sh.abs() * (w * sh.abs()).mean(1, keepdim=True)
    e_b = e_s * (w * sh.abs()).mean(1, keepdim=True) + sh.abs() * (w * e_s).mean(1, keepdim=True)
    bound = r.to(D)[:, None] * (DEPTH * U * mag + e_b) + 4 * U * wdx.abs() + 1e-30
    if dres is not None:
        bound = bound + 2 * U * dres.to(D).abs()
    if gt is BF:
        bound = bound + 2.0 ** -8 * wdx.abs()
    _within(dx, wdx, bound, "dx")
    ad = dy.to(D).abs()
    _within(dg, wdg, ((T + DEPTH) * U * (ad * sh.abs()) + ad * e_s).sum(0) + 1e-30, "dgamma")
    _within(db, wdb, (T + DEPTH) * U * ad.sum(0) + 1e-30, "dbeta")


def test_layer_norm_hard_rows(moe):
    """Constant rows, rows far from zero, tiny and huge rows, and rows with NaN
    or infinity, which must not reach their neighbours."""
    d = 2048
    g = _gen(5)
    x = torch.randn(9, d, generator=g)
    x[0] = 3.0                              # variance 0: y = beta
    x[1] = 0.0
    x[2] = 1000.0 + x[2]
    x[3] *= 1e-18
    x[4] *= 1e15
    x[5, 7] = float("nan")
    x[7, 0] = float("inf")
    beta = torch.randn(d, generator=g)
    _, y, mean, rstd = _run_norm(moe, x.to(DEV), None, None, beta.to(DEV))
    assert torch.equal(y[0].cpu(), beta.to(BF)) and torch.equal(y[1].cpu(), beta.to(BF))
    assert abs(rstd[0].item() - 1e-5 ** -0.5) < 1e-4 and mean[0].item() == 3.0
    ok = [2, 3, 4, 6, 8]
    wy, wm, wr, xh, e_mean, e_rstd, e_xh = _norm_bounds(x[ok], None, beta, 1e-5)
    _within(y[ok], wy, 2.0 ** -8 * wy.abs() + e_xh + 4 * U * beta.abs(), "y")
    assert torch.isnan(y[5]).all() and torch.isnan(y[7]).all()
    dy = torch.randn(9, d, generator=g).to(DEV)
    dx, dg, db = _run_norm_bwd(moe, x.to(DEV), dy, None, mean, rstd, None, FP)
    assert torch.isfinite(dx[[0, 1] + ok]).all() and torch.isnan(dx[5]).all()
    assert torch.isnan(dg).all()            # every column sums over the broken rows
    _within(db, dy.cpu().double().sum(0), 20 * U * dy.cpu().double().abs().sum(0), "dbeta")


def test_layer_norm_aliases_and_left_out_outputs(moe):
    """x_sum may be x and dx may be dres; statistics and weight gradients may
    be left out; none of it changes the bits."""
    g = _gen(6)
    n = lambda *s: torch.randn(*s, generator=g).to(DEV)
    T, d = 77, 1032
    x, add, dres = n(T, d).to(BF), n(T, d).to(BF), n(T, d).to(BF)
    gamma, beta, dy = n(d), n(d), n(T, d)
    x_sum, y, mean, rstd = _run_norm(moe, x, add, gamma, beta)
    xi, yi = x.clone(), torch.empty_like(y)
    moe.layer_norm(xi, add, gamma, beta, 1e-5, xi, yi, None, None)
    assert torch.equal(xi, x_sum) and torch.equal(yi, y)
    dx, dg, db = _run_norm_bwd(moe, x_sum, dy, gamma, mean, rstd, dres)
    buf = dres.clone()
    ws = torch.zeros(moe.layer_norm_backward_workspace_bytes(T, d), dtype=torch.uint8, device=DEV)
    moe.layer_norm_backward(x_sum, dy, gamma, mean, rstd, buf, buf, None, None, ws)
    assert torch.equal(buf, dx)
    only = torch.empty(d, device=DEV)
    moe.layer_norm_backward(x_sum, dy, gamma, mean, rstd, dres, buf, only, None, ws)
    assert torch.equal(only, dg)
    moe.layer_norm_backward(x_sum, dy, gamma, mean, rstd, dres, buf, None, only, ws)
    assert torch.equal(only, db)
    # no rows: weight gradients are zero
    e = torch.empty(0, d, device=DEV)
    dg0, db0 = torch.ones(d, device=DEV), torch.ones(d, device=DEV)
    moe.layer_norm_backward(e, e, gamma, e[:, 0], e[:, 0], None, e, dg0, db0, ws)
    assert not dg0.any() and not db0.any()


# ------------------------------------------------------------ balance loss --

def _run_balance(moe, logits, idx, mask, N, K, dlosses, dlogit):
    T = logits.shape[0]
    s = moe.Shape(T, 8, N, K, 8, 1)
    e = dict(device=DEV)
    out = dict(expert_count=torch.full((N,), -1, dtype=torch.int32, **e),
               token_count=torch.full((1,), -1, dtype=torch.int32, **e),
               expert_prob=torch.empty(N, **e), lse=torch.empty(T, **e), losses=torch.empty(2, **e),
               dlogits=torch.empty(T, N, **e))
    ws = torch.zeros(moe.balance_loss_workspace_bytes(s), dtype=torch.uint8, **e)
    moe.balance_loss(s, logits, idx, mask, out["expert_count"], out["token_count"],
                     out["expert_prob"], out["lse"], out["losses"], ws)
    moe.balance_loss_backward(s, logits, idx, mask, out["expert_count"], out["token_count"],
                              out["lse"], dlosses, dlogit, out["dlogits"])
    return out


def _check_balance(moe, logits, idx, mask, dlogit, dlosses=(0.7, 0.3)):
    T, N = logits.shape
    K = idx.shape[1]
    dl = torch.tensor(dlosses)
    dev = lambda t: None if t is None else t.to(DEV)
    got = _run_balance(moe, dev(logits), dev(idx), dev(mask), N, K, dl.to(DEV), dev(dlogit))
    want = ref.balance(logits, idx, mask, N)
    assert torch.equal(got["expert_count"].cpu().long(), want["expert_count"])
    assert int(got["token_count"]) == want["token_count"]
    # p: the exponential's argument is rounded at its own size (|l - lse| u),
    # expf and the division add a few u, the row's sum DEPTH u
    live = torch.ones(T, dtype=torch.bool) if mask is None else mask != 0
    fin = torch.where(torch.isfinite(logits) & live[:, None], logits, torch.zeros(())).to(D)
    size = fin.abs().amax() + math.log(N) + 1
    rel_p = (DEPTH + 4 * size) * U
    tc = max(want["token_count"], 1)
    _within(got["lse"][torch.isfinite(want["lse"]).to(DEV)], want["lse"][torch.isfinite(want["lse"])],
            (DEPTH + 4) * U * size, "lse")
    assert torch.equal(got["lse"].cpu() == -float("inf"), want["lse"] == -float("inf"))
    _within(got["expert_prob"], want["expert_prob"], (rel_p + (tc + DEPTH) * U) * want["expert_prob"] + 1e-30,
            "expert_prob")
    rel_l = torch.tensor([rel_p + (tc + N + DEPTH) * U, (tc + 2 * DEPTH) * U + 2 * (DEPTH + 4) * U * size],
                         dtype=D)
    _within(got["losses"], want["losses"], rel_l * (want["losses"].abs() + size ** 2 * torch.tensor([0.0, 1.0])) + 1e-30,
            "losses")
    wd = ref.balance_backward(logits, idx, mask, want["expert_count"], want["token_count"], dl, dlogit)
    f = want["expert_count"].to(D) / (tc * K)
    gate_only = torch.zeros(T, N, dtype=D)
    if dlogit is not None:
        gate_only = ref.balance_backward(logits, idx, torch.zeros(T), want["expert_count"], 0, dl, dlogit.abs())
    p = torch.zeros(T, N, dtype=D)
    use = torch.isfinite(want["lse"]) & live
    if use.any():
        p[use] = torch.softmax(logits[use].to(D), 1)
    mag = p * (dl[0] * N / tc * (f + (p @ f)[:, None]) + dl[1] * 2 / tc * want["lse"].nan_to_num(neginf=0.0).abs()[:, None])
    _within(got["dlogits"], wd, (2 * rel_p + (N + 2 * DEPTH) * U) * mag + 20 * U * gate_only + 1e-30, "dlogits")
    return got


@pytest.mark.parametrize("T,N,K", [(1, 1, 1), (1, 2, 1), (5, 3, 3), (64, 8, 2), (33, 31, 8),
                                   (200, 32, 4), (129, 33, 5), (500, 64, 8), (77, 128, 16),
                                   (90, 250, 8), (40, 255, 3), (61, 512, 6), (50, 1000, 16),
                                   (3000, 1024, 2), (20000, 16, 4)])
@pytest.mark.parametrize("masked", [False, True])
def test_balance_loss_and_gradient(moe, T, N, K, masked):
    g = _gen(T * 7 + N)
    logits = 2 * torch.randn(T, N, generator=g) + torch.randn(N, generator=g)
    idx = torch.topk(logits, K, 1).indices.int()
    mask = (torch.rand(T, generator=g) < 0.7).to(torch.uint8) * 3 if masked else None
    dlogit = None if masked else torch.randn(T, K, generator=g) / T
    _check_balance(moe, logits, idx, mask, dlogit)


@pytest.mark.parametrize("T,N,K", [(300, 1000, 16), (6000, 128, 8), (5000, 301, 4), (7886, 481, 1),
                                   (4000, 75, 14)])
def test_balance_many_partial_sums(moe, T, N, K):
    """Enough CTAs and experts that a cluster adds the partial sums, with fewer
    and more of them than its threads take at once; every call gives the same
    bits."""
    g = _gen(T + N)
    logits = 2 * torch.randn(T, N, generator=g)
    idx = torch.topk(logits + torch.randn(T, N, generator=g), K, 1).indices.int()
    dlogit = torch.randn(T, K, generator=g) / T
    got = _check_balance(moe, logits, idx, None, dlogit)
    again = _run_balance(moe, logits.to(DEV), idx.to(DEV), None, N, K, torch.tensor((0.7, 0.3)).to(DEV),
                         dlogit.to(DEV))
    for k in got:
        assert torch.equal(got[k], again[k]), k


@pytest.mark.parametrize("N", [1, 32, 34, 63, 64, 65, 66, 68, 95, 96, 97, 98, 100, 127, 129, 130, 132,
                               191, 192, 193, 194, 196, 257, 258, 260, 383, 384, 385, 386, 388,
                               511, 513, 514, 516])
def test_balance_row_widths(moe, N):
    """Either side of every width at which a row is held another way, for rows
    aligned to 4, 8 and 16 bytes; one row in the middle has a forbidden tail."""
    g = _gen(N)
    T, K = 67, min(N, 11)
    logits = 2 * torch.randn(T, N, generator=g)
    logits[40, N // 2 + 1:] = -float("inf")
    idx = torch.topk(logits + torch.randn(T, N, generator=g), K, 1).indices.int()
    _check_balance(moe, logits, idx, None, torch.randn(T, K, generator=g) / T)
    _check_balance(moe, logits, idx, None, None)


def test_balance_even_and_collapsed_routers(moe):
    """Even routing gives a loss of 1; a router that sends everything to one
    expert gives N (the extremes of the definition)."""
    T, N, K = 64, 8, 1
    idx = (torch.arange(T) % N).int()[:, None]
    got = _check_balance(moe, torch.zeros(T, N), idx, None, None)
    assert abs(got["losses"][0].item() - 1) < 1e-6
    assert abs(got["losses"][1].item() - math.log(N) ** 2) < 1e-5
    logits = torch.full((T, N), -100.0)
    logits[:, 3] = 0.0
    got = _check_balance(moe, logits, torch.full((T, 1), 3, dtype=torch.int32), None, None)
    assert abs(got["losses"][0].item() - N) < 1e-5


def test_balance_hard_rows(moe):
    """-inf logits, rows of nothing else, the lowest finite value, masked NaN,
    indices outside the experts and repeated ones, and no counted token."""
    T, N, K = 70, 40, 4
    g = _gen(8)
    logits = torch.randn(T, N, generator=g)
    idx = torch.topk(logits, K, 1).indices.int()
    logits[3, 5:] = -float("inf")
    logits[4] = -float("inf")
    logits[5, :39] = torch.finfo(torch.float32).min
    logits[6] = torch.finfo(torch.float32).min
    idx[8] = torch.tensor([-1, N, 2, 2 ** 31 - 1])
    idx[9] = 7                              # one expert four times
    dlogit = torch.randn(T, K, generator=g)
    # the lowest values dwarf every bound's size term: compare those rows on their own
    _check_balance(moe, torch.cat([logits[:5], logits[7:]]), torch.cat([idx[:5], idx[7:]]), None,
                   torch.cat([dlogit[:5], dlogit[7:]]))
    low = _run_balance(moe, logits[5:7].to(DEV), idx[5:7].to(DEV), None, N, K,
                       torch.tensor([1.0, 0.0], device=DEV), None)
    assert torch.isfinite(low["expert_prob"]).all()
    assert abs(low["expert_prob"][39].item() - (1 + 1 / N) / 2) < 1e-6
    assert torch.isfinite(low["dlogits"]).all()
    mask = torch.ones(T, dtype=torch.uint8)
    mask[10:30] = 0
    bad = logits.clone()
    bad[10:30] = float("nan")
    keep = [i for i in range(T) if i not in (5, 6)]
    _check_balance(moe, bad[keep], idx[keep], mask[keep], dlogit[keep])
    none = _check_balance(moe, bad[keep], idx[keep], torch.zeros(len(keep), dtype=torch.uint8), None)
    assert not none["losses"].any() and not none["dlogits"].any() and not none["expert_prob"].any()
    # a counted NaN or +inf is not hidden, and stays in its own row of the gradient
    for v in (float("nan"), float("inf")):
        broken = logits[7:].clone()
        broken[20, 3] = v
        out = _run_balance(moe, broken.to(DEV), idx[7:].to(DEV), None, N, K,
                           torch.tensor([1.0, 1.0], device=DEV), None)
        assert torch.isnan(out["losses"]).all()
        assert torch.isnan(out["dlogits"][20]).any()
        assert torch.isfinite(out["dlogits"][:20]).all() and torch.isfinite(out["dlogits"][21:]).all()


def test_balance_without_tokens(moe):
    s = moe.Shape(0, 8, 5, 2, 8, 1)
    e = dict(device=DEV)
    count, tok = torch.full((5,), 9, dtype=torch.int32, **e), torch.full((1,), 9, dtype=torch.int32, **e)
    prob, losses = torch.ones(5, **e), torch.ones(2, **e)
    ws = torch.zeros(moe.balance_loss_workspace_bytes(s), dtype=torch.uint8, **e)
    z = torch.empty(0, **e)
    moe.balance_loss(s, z, z.int(), None, count, tok, prob, z, losses, ws)
    assert not count.any() and not tok.any() and not prob.any() and not losses.any()


# ----------------------------------------------------- dense router gradient --

def _run_dense(moe, x, w, dl, dx_in, K=1):
    T, d = x.shape
    N = w.shape[0]
    s = moe.Shape(T, d, N, K, 8, 1)
    e = dict(device=DEV)
    dx, dw, db = torch.empty(T, d, **e), torch.empty(N, d, **e), torch.empty(N, **e)
    ws = torch.zeros(moe.router_dense_backward_workspace_bytes(s), dtype=torch.uint8, **e)
    moe.router_dense_backward(s, x, w, dl, dx_in, dx, dw, db, ws)
    assert moe.read_device_error(ws) == 0
    return dx, dw, db


@pytest.mark.parametrize("T,d,N", [(1, 8, 1), (3, 64, 2), (130, 72, 8), (257, 128, 33), (128, 256, 64),
                                   (1000, 264, 17), (700, 1000, 128), (129, 2048, 250),
                                   (300, 520, 512), (64, 136, 1024), (4100, 512, 32), (9000, 64, 5)])
@pytest.mark.parametrize("with_in", [True, False])
def test_router_dense_backward(moe, T, d, N, with_in):
    """fp32 products: each sum of n terms within 2 n u of its terms' size (the
    factor covers operands held as sums of shorter pieces), and over the whole
    output within 2e-5 in the 2-norm, some 30 u times the square root of the
    longest sum here."""
    g = _gen(T + 3 * d + N)
    n = lambda *s: torch.randn(*s, generator=g)
    x, w, dl = n(T, d).to(BF), 0.02 * n(N, d), n(T, N) * torch.exp(2 * n(T, 1))
    dx_in = n(T, d) if with_in else None
    dx, dw, db = _run_dense(moe, x.to(DEV), w.to(DEV), dl.to(DEV), dx_in.to(DEV) if with_in else None)
    a, b, c = dl.double(), w.double(), x.double()
    base = dx_in.double() if with_in else torch.zeros(T, d, dtype=D)
    for got, want, size, k, what in ((dx, base + a @ b, base.abs() + a.abs() @ b.abs(), N, "dx"),
                                     (dw, a.t() @ c, a.abs().t() @ c.abs(), T, "dw_router"),
                                     (db, a.sum(0), a.abs().sum(0), T, "dbias")):
        _within(got, want, (2 * k + 64) * U * size + 1e-30, what)
        assert (got.cpu().double() - want).norm() <= 2e-5 * want.norm(), what


def test_router_dense_backward_wide_range(moe):
    """Entries from 1e-30 to 1e30, and the largest fp32 values, keep fp32
    accuracy (a piece that is rounded away or overflows would show)."""
    g = _gen(11)
    T, d, N = 200, 64, 24
    n = lambda *s: torch.randn(*s, generator=g)
    x = torch.ones(T, d).to(BF)
    for scale_dl, scale_w in ((1e-30, 1.0), (1e30, 1e-30), (1e-18, 1e18), (3.4e38, 1e-3)):
        w = n(N, d).clamp(-1, 1) * scale_w
        dl = torch.zeros(T, N)
        dl[torch.arange(T), torch.arange(T) % N] = n(T).clamp(-1, 1).sign() * scale_dl
        dx, dw, db = _run_dense(moe, x.to(DEV), w.to(DEV), dl.to(DEV), None)
        want = dl.double() @ w.double()
        _within(dx, want, 64 * U * want.abs() + 1e-36, f"dx at {scale_dl}")


def test_router_dense_backward_left_out_and_in_place(moe):
    g = _gen(12)
    T, d, N = 300, 264, 40
    s = moe.Shape(T, d, N, 1, 8, 1)
    x, w, dl, base = (torch.randn(*q, generator=g).to(DEV) for q in ((T, d), (N, d), (T, N), (T, d)))
    x = x.to(BF)
    dx, dw, db = _run_dense(moe, x, w, dl, base)
    ws = torch.zeros(moe.router_dense_backward_workspace_bytes(s), dtype=torch.uint8, device=DEV)
    buf = base.clone()
    moe.router_dense_backward(s, x, w, dl, buf, buf, None, None, ws)
    assert torch.equal(buf, dx)
    o = torch.empty(N, d, device=DEV)
    moe.router_dense_backward(s, x, w, dl, None, None, o, None, ws)
    assert torch.equal(o, dw)
    o = torch.empty(N, device=DEV)
    moe.router_dense_backward(s, None, None, dl, None, None, None, o, ws)
    assert torch.equal(o, db)
    # no tokens: weight gradients are zero
    s0 = moe.Shape(0, d, N, 1, 8, 1)
    z = torch.empty(0, device=DEV)
    dw0, db0 = torch.ones(N, d, device=DEV), torch.ones(N, device=DEV)
    ws0 = torch.zeros(moe.router_dense_backward_workspace_bytes(s0), dtype=torch.uint8, device=DEV)
    moe.router_dense_backward(s0, z.to(BF), w, z, None, z, dw0, db0, ws0)
    assert not dw0.any() and not db0.any()


@pytest.mark.parametrize("T,d,N", [(9000, 64, 5), (2500, 128, 24), (85, 328, 381), (40, 4096, 64)])
def test_router_dense_weight_gradients_do_not_depend_on_dx(moe, T, d, N):
    """Many partial sums of few weights and few of many, with more and fewer
    tiles of dx than CTAs that add them: the same bits with and without dx."""
    g = _gen(T + d + N)
    n = lambda *q: torch.randn(*q, generator=g).to(DEV)
    x, w, dl, base = n(T, d).to(BF), n(N, d), n(T, N), n(T, d)
    s = moe.Shape(T, d, N, 1, 8, 1)
    _, dw, db = _run_dense(moe, x, w, dl, base)
    ws = torch.zeros(moe.router_dense_backward_workspace_bytes(s), dtype=torch.uint8, device=DEV)
    o, ob = torch.full_like(dw, float("nan")), torch.full_like(db, float("nan"))
    moe.router_dense_backward(s, x, None, dl, None, None, o, ob, ws)
    assert torch.equal(o, dw) and torch.equal(ob, db)


def test_router_dense_backward_non_finite(moe):
    """A broken token's gradient does not reach other tokens' dx; it reaches
    dw_router's rows of its broken logits only where x is finite."""
    g = _gen(13)
    T, d, N = 260, 128, 24
    x, w, dl = (torch.randn(*q, generator=g).to(DEV) for q in ((T, d), (N, d), (T, N)))
    x = x.to(BF)
    good = _run_dense(moe, x, w, dl, None)
    for v in (float("nan"), float("inf")):
        bad = dl.clone()
        bad[130, 5] = v
        dx, dw, db = _run_dense(moe, x, w, bad, None)
        assert not torch.isfinite(dx[130]).any()
        rest = [t for t in range(T) if t != 130]
        assert torch.equal(dx[rest], good[0][rest])
        assert not torch.isfinite(dw[5]).any() and not torch.isfinite(db[5])
        others = [e for e in range(N) if e != 5]
        assert torch.equal(dw[others], good[1][others]) and torch.equal(db[others], good[2][others])


# ------------------------------------------------------- 8-bit checkpoints --

def _packed(T, N, K, cap, g, skew=0.0):
    """A route map as moe_route packs it: rows, counts, offsets."""
    score = torch.rand(T, N, generator=g) ** (1 + skew * torch.arange(N))
    idx = torch.topk(score, K, 1).indices
    hot = torch.zeros(T, N, dtype=torch.int64).scatter(1, idx, 1)
    rank = (torch.cumsum(hot, 0) - hot).gather(1, idx)
    count = hot.sum(0).clamp(max=cap)
    off = torch.zeros(N + 1, dtype=torch.int64)
    off[1:] = torch.cumsum(count, 0)
    row = torch.where(rank < cap, off[idx] + rank, -1)
    return row.int(), off.int()


def _run_checkpoint(moe, s, off, g, u, y, fill=7):
    R, h, d = s.R, s.h, s.d
    e = dict(device=DEV)
    q = {n: (torch.full((R, c), fill, dtype=torch.int8, **e),
             torch.full((R, c // 32), fill, dtype=torch.uint8, **e))
         for n, c in (("g", h), ("u", h), ("y", d))}
    moe.checkpoint_save(s, off, g, u, y, *q["g"], *q["u"], *q["y"])
    out = [torch.full((R, h), float(fill), dtype=BF, **e) for _ in range(3)]
    moe.checkpoint_restore(s, off, *q["g"], *q["u"], *out)
    return q, out


@pytest.mark.parametrize("T,d,N,K,h,cap", [(1, 32, 1, 1, 32, 1), (5, 64, 3, 2, 96, 2), (64, 128, 8, 2, 256, 20),
                                           (300, 160, 16, 4, 64, 60), (129, 2048, 9, 8, 32, 129),
                                           (700, 96, 5, 5, 1024, 350), (40, 32, 4, 2, 32, 0)])
def test_checkpoint_codes_values_and_backward(moe, T, d, N, K, h, cap):
    """Codes, scales and restored values bit for bit; rows past the packed
    ones untouched; the combine backward against 64 bits: dy_disp is one fp32
    product rounded once (bit-exact), dgate a sum of d terms."""
    gen = _gen(T + d + h)
    row, off = _packed(T, N, K, cap, gen, 0.2)
    s = moe.Shape(T, d, N, K, h, cap)
    R, Acc = s.R, int(off[-1])
    mk = lambda c: (torch.randn(R, c, generator=gen) * torch.exp(4 * torch.randn(R, 1, generator=gen))).to(BF)
    g, u, y = mk(h), mk(h), mk(d)
    for t in (g, u, y):
        if R > 2:
            t[Acc // 2, :32] = 0.0                      # a block of zeros
            t[Acc // 3, :32] *= 0.0
            t[Acc // 3, 3] = 2.0 ** -130                # subnormal only
        t[Acc:] = float("nan")                          # the tail holds anything
    dy, gate = torch.randn(T, d, generator=gen).to(BF), torch.rand(T, K, generator=gen)
    q, out = _run_checkpoint(moe, s, off.to(DEV), g.to(DEV), u.to(DEV), y.to(DEV))
    vals = {}
    for n, t in (("g", g), ("u", u), ("y", y)):
        wq, ws = ref.mxint8(t[:Acc])
        assert torch.equal(q[n][0][:Acc].cpu(), wq) and torch.equal(q[n][1][:Acc].cpu(), ws), n
        assert (q[n][0][Acc:] == 7).all() and (q[n][1][Acc:] == 7).all(), n
        vals[n] = ref.mxint8_value(wq, ws)
    for o, n in ((out[0], "g"), (out[1], "u")):
        assert torch.equal(o[:Acc].cpu().double(), vals[n]), n
    wh = vals["g"] * torch.sigmoid(vals["g"]) * vals["u"]
    # __expf is good to 2 + |1.16 x| ulp of its result, past |x| = 88 the
    # sigmoid is 0 or 1 (or the product has left the normal range)
    lim = (2.0 ** -8 + 300 * U) * wh.abs() + 2.0 ** -126 * (1 + vals["u"].abs())
    _within(out[2][:Acc], wh, lim, "h_act")
    for o in out:
        assert (o[Acc:] == 7).all()
    dyd = torch.full((R, d), 7.0, dtype=BF, device=DEV)
    dgate, dlogit = torch.empty(T, K, device=DEV), torch.empty(T, K, device=DEV)
    moe.combine_backward_checkpoint(s, dy.to(DEV), *q["y"], row.to(DEV), gate.to(DEV), dyd, dgate, dlogit)
    wdy = torch.full((R, d), 7.0, dtype=BF)
    wdg, mag = torch.zeros(T, K, dtype=D), torch.zeros(T, K, dtype=D)
    for k in range(K):
        t = torch.nonzero(row[:, k] >= 0)[:, 0]
        r = row[t, k].long()
        wdy[r] = (gate[t, k][:, None] * dy[t].float()).to(BF)
        wdg[t, k] = (dy[t].double() * vals["y"][r]).sum(1)
        mag[t, k] = (dy[t].double() * vals["y"][r]).abs().sum(1)
    assert torch.equal(dyd.cpu(), wdy)
    _within(dgate, wdg, (d + 8) * U * mag, "dgate")
    # the gates' Jacobian takes the dgate that was written (K <= 16 fp32 terms)
    dg, gg = dgate.cpu().double(), gate.double()
    dot = (gg * dg).sum(1, keepdim=True)
    size = gg * (dg.abs() + (gg * dg).abs().sum(1, keepdim=True))
    _within(dlogit, gg * (dg - dot), 20 * U * size + 1e-30, "dlogit")
    alone = torch.empty(T, K, device=DEV)
    moe.combine_backward_checkpoint(s, dy.to(DEV), *q["y"], row.to(DEV), gate.to(DEV), dyd, alone)
    assert torch.equal(alone, dgate)


def test_checkpoint_every_bf16_value(moe):
    """Every bf16 bit pattern, as the largest of a block and beside smaller
    ones: codes and scales bit for bit, NaN and infinity as a whole block."""
    allv = torch.arange(-32768, 32768, dtype=torch.int32).to(torch.int16).view(BF)
    blocks = torch.zeros(65536, 32, dtype=BF)
    blocks[:, 0] = allv
    blocks[:, 1:] = (allv.float()[:, None] * torch.linspace(-1, 1, 31)[None]).to(BF)
    big = ~torch.isfinite(allv.float())
    blocks[big, 2:] = 1.0
    R = 65536
    s = moe.Shape(R, 32, 1, 1, 32, R)
    off = torch.tensor([0, R], dtype=torch.int32, device=DEV)
    q, out = _run_checkpoint(moe, s, off, blocks.to(DEV), blocks.to(DEV), blocks.to(DEV))
    wq, ws = ref.mxint8(blocks)
    for n in "guy":
        assert torch.equal(q[n][0].cpu(), wq) and torch.equal(q[n][1].cpu(), ws), n
    v = ref.mxint8_value(wq, ws)
    assert torch.equal(torch.isnan(out[0]).cpu(), torch.isnan(v))
    assert torch.equal(out[0].cpu().double().nan_to_num(1.5), v.nan_to_num(1.5))


def test_checkpoint_sources_left_out(moe):
    T, d, N, K, h, cap = 50, 64, 4, 2, 96, 20
    gen = _gen(21)
    row, off = _packed(T, N, K, cap, gen)
    s = moe.Shape(T, d, N, K, h, cap)
    e = dict(device=DEV)
    y = torch.randn(s.R, d, generator=gen).to(BF).to(DEV)
    yq, ys = torch.zeros(s.R, d, dtype=torch.int8, **e), torch.zeros(s.R, d // 32, dtype=torch.uint8, **e)
    moe.checkpoint_save(s, off.to(DEV), None, None, y, None, None, None, None, yq, ys)
    wq, ws = ref.mxint8(y.cpu()[:int(off[-1])])
    assert torch.equal(yq.cpu()[:int(off[-1])], wq) and torch.equal(ys.cpu()[:int(off[-1])], ws)


# -------------------------------------------------- streams, graphs, length --

def _one_of_each(moe, seed=3):
    """A closure that runs every operator on fixed buffers, and its outputs."""
    gen = _gen(seed)
    n = lambda *s: torch.randn(*s, generator=gen).to(DEV)
    T, d, N, K, h, cap = 300, 256, 16, 2, 64, 45
    s = moe.Shape(T, d, N, K, h, cap)
    x, add, dy, dres = n(T, d).to(BF), n(T, d).to(BF), n(T, d), n(T, d).to(BF)
    gamma, beta, logits, w = n(d), n(d), n(T, N), n(N, d)
    idx = torch.topk(logits, K, 1).indices.int()
    row, off = (t.to(DEV) for t in _packed(T, N, K, cap, gen))
    g, u, y = n(s.R, h).to(BF), n(s.R, h).to(BF), n(s.R, d).to(BF)
    gate, dlosses = torch.rand(T, K, generator=gen).to(DEV), n(2)
    z = lambda *q, dt=FP: torch.zeros(*q, dtype=dt, device=DEV)
    o = dict(x_sum=z(T, d, dt=BF), y=z(T, d, dt=BF), mean=z(T), rstd=z(T), dx=z(T, d, dt=BF),
             dgamma=z(d), dbeta=z(d), count=z(N, dt=torch.int32), tok=z(1, dt=torch.int32), prob=z(N),
             lse=z(T), losses=z(2), dlogits=z(T, N), rdx=z(T, d), rdw=z(N, d), rdb=z(N),
             gq=z(s.R, h, dt=torch.int8), gs=z(s.R, h // 32, dt=torch.uint8),
             uq=z(s.R, h, dt=torch.int8), us=z(s.R, h // 32, dt=torch.uint8),
             yq=z(s.R, d, dt=torch.int8), ys=z(s.R, d // 32, dt=torch.uint8),
             g=z(s.R, h, dt=BF), u=z(s.R, h, dt=BF), h=z(s.R, h, dt=BF), dyd=z(s.R, d, dt=BF),
             dgate=z(T, K))
    w8 = lambda b: torch.zeros(b, dtype=torch.uint8, device=DEV)
    ws = [w8(moe.layer_norm_backward_workspace_bytes(T, d)), w8(moe.balance_loss_workspace_bytes(s)),
          w8(moe.router_dense_backward_workspace_bytes(s))]

    def run(stream=None):
        moe.layer_norm(x, add, gamma, beta, 1e-5, o["x_sum"], o["y"], o["mean"], o["rstd"], stream=stream)
        moe.layer_norm_backward(o["x_sum"], dy, gamma, o["mean"], o["rstd"], dres, o["dx"], o["dgamma"],
                                o["dbeta"], ws[0], stream=stream)
        moe.balance_loss(s, logits, idx, None, o["count"], o["tok"], o["prob"], o["lse"], o["losses"],
                         ws[1], stream=stream)
        moe.balance_loss_backward(s, logits, idx, None, o["count"], o["tok"], o["lse"], dlosses, gate,
                                  o["dlogits"], stream=stream)
        moe.router_dense_backward(s, o["y"], w, o["dlogits"], dy, o["rdx"], o["rdw"], o["rdb"], ws[2],
                                  stream=stream)
        moe.checkpoint_save(s, off, g, u, y, o["gq"], o["gs"], o["uq"], o["us"], o["yq"], o["ys"],
                            stream=stream)
        moe.combine_backward_checkpoint(s, dres, o["yq"], o["ys"], row, gate, o["dyd"], o["dgate"],
                                        stream=stream)
        moe.checkpoint_restore(s, off, o["gq"], o["gs"], o["uq"], o["us"], o["g"], o["u"], o["h"],
                               stream=stream)
    return run, o


def test_same_bits_on_every_run_stream_and_in_a_graph(moe):
    run, o = _one_of_each(moe)
    run()
    torch.cuda.synchronize()
    first = {k: v.clone() for k, v in o.items()}

    def same():
        for k in o:
            assert torch.equal(o[k], first[k]), k
            o[k].zero_()
        torch.cuda.synchronize()

    for _ in range(3):
        run()
    torch.cuda.synchronize()
    same()
    side = torch.cuda.Stream()
    run(stream=side)                        # an explicit stream, not the current one
    side.synchronize()
    same()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run()
    for v in o.values():
        v.zero_()
    graph.replay()
    torch.cuda.synchronize()
    same()


def test_no_host_synchronisation(moe):
    run, o = _one_of_each(moe)
    run()
    torch.cuda.synchronize()
    torch.cuda.set_sync_debug_mode("error")
    try:
        run()
    finally:
        torch.cuda.set_sync_debug_mode("default")
    torch.cuda.synchronize()


def _last_rows_equal(big, small, k):
    assert torch.equal(big[-k:], small), "the last rows differ from the same rows alone"


def test_offsets_past_32_bits(moe):
    """Buffers of more than 2^31 elements: the last rows of one long call equal
    the same rows in a call of their own."""
    k, d = 16, 8192
    T = (1 << 31) // d + 40
    x = torch.zeros(T, d, dtype=BF, device=DEV)
    x[-k:] = torch.randn(k, d, generator=_gen(31)).to(BF).to(DEV)
    y = torch.empty_like(x)
    st = [torch.empty(T, device=DEV) for _ in range(2)]
    moe.layer_norm(x, None, None, None, 1e-5, None, y, *st)
    _, ys, ms, rs = _run_norm(moe, x[-k:].clone(), None, None, None)
    _last_rows_equal(y, ys, k)
    _last_rows_equal(st[0], ms, k)
    ws = torch.zeros(moe.layer_norm_backward_workspace_bytes(T, d), dtype=torch.uint8, device=DEV)
    dx = torch.empty_like(x)
    moe.layer_norm_backward(x, y, None, st[0], st[1], x, dx, None, None, ws)
    dxs, _, _ = _run_norm_bwd(moe, x[-k:].clone(), ys, None, ms, rs, x[-k:].clone(), weights=False)
    _last_rows_equal(dx, dxs, k)
    # checkpoints of one expert's rows
    s, ss = moe.Shape(T, 32, 1, 1, d, T), moe.Shape(k, 32, 1, 1, d, k)
    off = torch.tensor([0, T], dtype=torch.int32, device=DEV)
    offs = torch.tensor([0, k], dtype=torch.int32, device=DEV)
    q = torch.zeros(T, d, dtype=torch.int8, device=DEV)
    sc = torch.zeros(T, d // 32, dtype=torch.uint8, device=DEV)
    moe.checkpoint_save(s, off, x, None, None, q, sc, None, None, None, None)
    wq, wsc = ref.mxint8(x[-k:].cpu())
    _last_rows_equal(q.cpu(), wq, k)
    _last_rows_equal(sc.cpu(), wsc, k)
    moe.checkpoint_restore(s, off, q, sc, q, sc, y, dx, x)
    small = [torch.empty(k, d, dtype=BF, device=DEV) for _ in range(3)]
    moe.checkpoint_restore(ss, offs, wq.to(DEV), wsc.to(DEV), wq.to(DEV), wsc.to(DEV), *small)
    for a, b in zip((y, dx, x), small):
        _last_rows_equal(a, b, k)
    del x, y, dx, q, sc
    torch.cuda.empty_cache()
    N = 1024
    T = (1 << 31) // N + 40
    logits = torch.zeros(T, N, device=DEV)
    logits[-k:] = torch.randn(k, N, generator=_gen(32)).to(DEV)
    idx = torch.arange(T, dtype=torch.int32, device=DEV)[:, None] % N
    out = _run_balance(moe, logits, idx, None, N, 1, torch.tensor([1.0, 1.0], device=DEV), None)
    assert int(out["token_count"]) == T and int(out["expert_count"].sum()) == T
    p = torch.softmax(logits[-k:].double(), 1)
    f = out["expert_count"].double() / T
    lse = torch.logsumexp(logits[-k:].double(), 1, keepdim=True)
    want = p * (N / T * (f - (p @ f)[:, None]) + 2 / T * lse)
    assert (out["dlogits"][-k:].double() - want).norm() <= 1e-4 * want.norm()


def test_router_dense_offsets_past_32_bits(moe):
    """More than 2^31 elements in x, dx_in and dx: the last tokens' dx equals the
    same tokens' in a call of their own, and dw_router is theirs alone when every
    other token is zero."""
    k, d, N = 200, 8192, 6
    T = (1 << 31) // d + 72
    g = _gen(33)
    x, dl = torch.zeros(T, d, dtype=BF, device=DEV), torch.zeros(T, N, device=DEV)
    x[-k:] = torch.randn(k, d, generator=g).to(BF).to(DEV)
    dl[-k:] = torch.randn(k, N, generator=g).to(DEV)
    w = torch.randn(N, d, generator=g).to(DEV)
    dx = torch.zeros(T, d, device=DEV)
    dx[-k:] = torch.randn(k, d, generator=g).to(DEV)
    base = dx[-k:].clone()
    s = moe.Shape(T, d, N, 1, 8, 1)
    dw, db = torch.empty(N, d, device=DEV), torch.empty(N, device=DEV)
    ws = torch.zeros(moe.router_dense_backward_workspace_bytes(s), dtype=torch.uint8, device=DEV)
    moe.router_dense_backward(s, x, w, dl, dx, dx, dw, db, ws)
    assert moe.read_device_error(ws) == 0
    sdx, sdw, sdb = _run_dense(moe, x[-k:].clone(), w, dl[-k:].clone(), base)
    _last_rows_equal(dx, sdx, k)
    assert not dx[: 1 << 12].any() and not dx[(1 << 31) // d - 4096:-k].any()
    assert torch.allclose(dw, sdw, rtol=1e-5, atol=1e-4) and torch.allclose(db, sdb, rtol=1e-5, atol=1e-4)
