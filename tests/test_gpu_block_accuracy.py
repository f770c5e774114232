"""Accuracy of the block operators where a long sum, a large common value or a
loop's later rounds would show it, on the GPU against 64 bits.

u = 2^-24 is the unit roundoff of fp32."""
import pytest
import torch

import _block_ref as ref
import test_gpu_block as block
from _gpu_util import DEV

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
BF, FP, D = torch.bfloat16, torch.float32, torch.float64
LOWEST = torch.finfo(torch.float32).min


@pytest.fixture(scope="module")
def moe():
    import __graft_entry__
    __graft_entry__.build()
    import combine_expert_gemm_gb300 as m
    return m


# ------------------------------------------------------------ balance loss --

@pytest.mark.parametrize("offset", [0.0, 100.0, -100.0, 1e4, -1e7, 1e9, -1e9, 3e38, LOWEST])
@pytest.mark.parametrize("N,K", [(24, 2), (64, 8), (90, 3), (128, 8), (161, 4), (250, 8), (384, 6), (500, 4),
                                 (1000, 8)])
def test_balance_gradient_does_not_depend_on_a_common_value(moe, N, K, offset):
    """p is a softmax: a value common to a row's logits changes nothing but
    which fp32 values the logits round to (at 1e9 they round to multiples of
    64, at the lowest value all to one).  So the bound holds no size of the
    logits, only `spread`, how far the row's other logits lie below its largest.

    p: the exponential's argument takes three roundings of at most spread +
    log N + 1, the exponential and the division 4 u each, the row's sum one u
    for each of at most 32 + 5 levels; the product with f and its sum as much
    again.  A few u for the rest: (6 size + 160) u of the terms."""
    g = torch.Generator().manual_seed(N)
    T = 83
    base = 2 * torch.randn(T, N, generator=g)
    logits = torch.full((T, N), LOWEST) if offset == LOWEST else base + offset
    if offset != LOWEST:
        logits[7, N // 2:] = -float("inf")
        logits[8, 1:] = LOWEST
    idx = torch.topk(base + torch.randn(N, generator=g), K, 1).indices.int()
    dlosses = torch.tensor([0.7, 0.0])
    got = block._run_balance(moe, logits.to(DEV), idx.to(DEV), None, N, K, dlosses.to(DEV), None)
    count = torch.bincount(idx.reshape(-1).long(), minlength=N)
    assert torch.equal(got["expert_count"].cpu().long(), count)
    want = ref.balance_backward(logits, idx, None, count, T, dlosses, None)
    p = torch.softmax(logits.to(D), 1)
    f = count.to(D) / (T * K)
    spread = torch.where(p > 0, logits.to(D).amax(1, keepdim=True) - logits.to(D), 0.0).clamp(max=100).amax()
    size = spread + torch.log(torch.tensor(float(N))) + 1
    mag = p * (0.7 * N / T) * (f + (p @ f)[:, None])
    block._within(got["dlogits"], want, (6 * size + 160) * U * mag + 1e-30, "dlogits")
    block._within(got["expert_prob"], p.mean(0), (3 * size + 160 + T) * U * p.mean(0) + 1e-30, "expert_prob")


@pytest.mark.parametrize("m", [0.0, 0.02, -0.02])
def test_balance_log_sum_of_nearly_certain_rows(moe, m):
    """log sum e of rows with one expert far ahead, whose log of the sum 1 +
    e^-d is itself near 0: no absolute error of a short logarithm hides there.
    The sum is rounded by u, its second term by (3 d + 4) u of itself, the
    logarithm by 2 u of itself and the result by u of itself."""
    T, N = 20000, 2
    g = torch.Generator().manual_seed(3)
    d = 3 + 9 * torch.rand(T, generator=g)
    logits = torch.stack([torch.full((T,), m), m - d], 1)
    idx = torch.zeros(T, 1, dtype=torch.int32)
    got = block._run_balance(moe, logits.to(DEV), idx.to(DEV), None, N, 1, torch.tensor([1.0, 1.0], device=DEV), None)
    want = torch.logsumexp(logits.to(D), 1)
    d = (logits[:, 0].to(D) - logits[:, 1].to(D))
    block._within(got["lse"], want, U * (1.1 + (3 * d + 6) * torch.exp(-d) + want.abs()), "lse")


def test_balance_sums_over_warps_are_trees(moe):
    """One token's square of 1 and 31 of 2^-25, each in a warp of its own: added
    one after the other to the 1 they all vanish (15 u).  A tree over lanes and
    warps rounds once a level, at most 5 + 5 + 2 u."""
    T = 128                                    # four tokens of one expert a warp, 32 warps
    logits = torch.zeros(T, 1)
    logits[::4] = 2.0 ** -12.5
    logits[0] = 1.0
    got = block._run_balance(moe, logits.to(DEV), torch.zeros(T, 1, dtype=torch.int32, device=DEV), None, 1, 1,
                             torch.tensor([1.0, 1.0], device=DEV), None)
    want = (logits.to(D) ** 2).sum() / T
    assert abs(got["losses"][1].double().item() - want.item()) <= 12 * U * want.item()
    assert got["losses"][0].item() == 1.0


# ----------------------------------------------------- dense router gradient --

def _chain(a, b):
    """a @ b as fp32 products are summed: one fused multiply-add after the other."""
    out = torch.zeros(a.shape[0], b.shape[1], device=a.device)
    for k in range(a.shape[1]):
        # the product is exact in 64 bits, the sum is rounded once more there
        out = (out.double() + a[:, k, None].double() * b[k, None].double()).float()
    return out


def _as_good_as_fp32(got, a, b, what):
    """Within twice the chain's error and 5 u in the 2-norm.  The second term
    is for sums so short that the chain hardly rounds: a k-block's partial sum
    is cut, not rounded, and loses at most one unit in the last place, 2 u, in
    each of its last two steps, and the pieces hold each operand to u / 2.  The
    factor covers that the order of the sum is another one."""
    want = a.double() @ b.double()
    err = lambda t: ((t.double() - want).norm() / want.norm()).item()
    mine, chain = err(got), err(_chain(a, b))
    assert mine <= 2 * chain + 5 * U, f"{what}: {mine:.3g}, an fp32 chain {chain:.3g}"


@pytest.mark.parametrize("sign", ["mixed", "same"])
@pytest.mark.parametrize("T,d,N", [(300, 264, 8), (300, 264, 32), (333, 264, 48), (333, 264, 64), (400, 264, 100),
                                   (500, 520, 128), (257, 1032, 250), (700, 264, 256), (300, 520, 512),
                                   (150, 1544, 1000), (200, 264, 1024), (64, 2048, 300), (2100, 136, 64)])
def test_router_dense_keeps_fp32_accuracy(moe, T, d, N, sign):
    """Every expert count from one k-block of dx to 32 of them: the error of an
    fp32 product of the same length, without dx_in to hide it.  Operands of one
    sign show a sum that drifts, of both signs one that loses pieces."""
    g = torch.Generator().manual_seed(T + N)
    n = lambda *s: torch.randn(*s, generator=g)
    x, w, dl = n(T, d).to(BF).float(), n(N, d), n(T, N)
    if sign == "same":
        x, w, dl = x.abs(), w.abs(), dl.abs()
    x, w, dl = x.to(DEV), w.to(DEV), dl.to(DEV)
    dx, dw, db = block._run_dense(moe, x.to(BF), w, dl, None)
    _as_good_as_fp32(dx, dl, w, "dx")
    _as_good_as_fp32(dw, dl.t().contiguous(), x, "dw_router")
    _as_good_as_fp32(db[:, None], dl.t().contiguous(), torch.ones(T, 1, device=DEV), "dbias")


@pytest.mark.parametrize("N", [8, 40, 200, 600])
def test_router_dense_products_of_single_entries(moe, N):
    """One token for each expert and full 24-bit values: each element is one
    product.  dw_router's is exact but for one cut (2 u); dx's leaves out piece
    products below 2^-24, 2^-24 and 2^-32 of it and is cut at most four times;
    dbias is the value itself."""
    g = torch.Generator().manual_seed(N)
    d = 72
    n = lambda *s: torch.randn(*s, generator=g)
    x = n(N, d).to(BF)
    for scale_dl, scale_w in ((1.0, 1.0), (1e-30, 1e6), (1e30, 1e-30), (1e-18, 1e18), (1e36, 1e-3)):
        v, w = n(N) * scale_dl, n(N, d) * scale_w
        dl = torch.diag(v)
        dx, dw, db = block._run_dense(moe, x.to(DEV), w.to(DEV), dl.to(DEV), None)
        assert torch.equal(db.cpu(), v)
        want = v.double()[:, None] * x.double()
        block._within(dw, want, 4 * U * want.abs() + 1e-37, f"dw at {scale_dl}")
        want = v.double()[:, None] * w.double()
        block._within(dx, want, 12 * U * want.abs() + 1e-37, f"dx at {scale_dl}")


@pytest.mark.parametrize("T,d,N", [(8192, 2048, 64), (9001, 4104, 31), (5000, 3080, 100), (6000, 2568, 200),
                                   (4097, 1992, 1000), (40000, 264, 5)])
@pytest.mark.parametrize("with_in", [True, False])
def test_router_dense_later_rounds(moe, T, d, N, with_in):
    """Enough tiles and k-blocks that every ring, accumulator and slot of a CTA
    is used several times over, and every CTA that splits dlogits has more than
    one block of tokens in the cases that can: dense data, so that a block
    taken twice, left out or stale would show.  The bounds are those of
    sums of n terms (2 n u), and the chain's in the 2-norm."""
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    tiles, k_blocks = -(-T // 128) * -(-d // 128), -(-N // 32)
    assert tiles >= 6 * sms or tiles * k_blocks >= 48 * sms or T >= 38912   # rounds of dx, or of the split
    g = torch.Generator(device=DEV).manual_seed(T + N)
    n = lambda *s: torch.randn(*s, generator=g, device=DEV)
    x, w, dl = n(T, d).to(BF), 0.02 * n(N, d), n(T, N)
    dx_in = n(T, d) if with_in else None
    dx, dw, db = block._run_dense(moe, x, w, dl, dx_in)
    a, b, c = dl.double(), w.double(), x.double()
    base = dx_in.double() if with_in else torch.zeros_like(c)
    for got, want, size, k, what in ((dx, base + a @ b, base.abs() + a.abs() @ b.abs(), N, "dx"),
                                     (dw, a.t() @ c, a.abs().t() @ c.abs(), T, "dw_router"),
                                     (db, a.sum(0), a.abs().sum(0), T, "dbias")):
        off = (got.double() - want).abs() - (2 * k + 64) * U * size
        assert not (off > 0).any(), what
    if not with_in:
        _as_good_as_fp32(dx, dl, w, "dx")
        rows = slice(0, 5)                     # the chain over T on a few experts
        _as_good_as_fp32(dw[rows], dl[:, rows].t().contiguous(), x.float(), "dw_router")


# -------------------------------------------------------------- layer norm --

@pytest.mark.parametrize("T,d,xt,yt,gt", [
    (30001, 64, BF, FP, BF), (26001, 256, FP, BF, FP), (8195, 2048, BF, FP, BF), (3300, 4096, FP, BF, BF),
    (8000, 1032, FP, FP, FP), (1700, 8192, BF, BF, BF), (1601, 8200, FP, FP, BF), (1700, 16376, BF, FP, FP),
])
@pytest.mark.parametrize("kind", ["full", "bare"])
def test_layer_norm_many_rows_a_group(moe, T, d, xt, yt, gt, kind):
    """At least ten rows for each group of warps, so that the copies' ring, the
    alternating buffers of the row sums and the weight gradients' registers are
    used over and over, with the bounds of the short cases."""
    warps = -(-d // 512)                       # of a group, at 16 columns a thread
    groups = max(1, 16 // warps) * torch.cuda.get_device_properties(0).multi_processor_count
    assert T >= 10 * groups
    block.test_layer_norm_and_backward(moe, T, d, xt, yt, gt, kind)
