"""The dense operators at the ends of their ranges: sums of squares that leave fp32,
long sums, and what is refused.  The bounds are those of test_gpu_dense.py unless a
test states its own."""
import pytest
import torch

import _dense_ref as ref
from _gpu_util import DEV
from test_gpu_dense import _check_ns, _mats, _ns, _ns_bound, _ws

pytestmark = pytest.mark.gpu
BF, FP, D = torch.bfloat16, torch.float32, torch.float64


@pytest.fixture(scope="module")
def moe():
    import __graft_entry__
    __graft_entry__.build()
    import combine_expert_gemm_gb300 as m
    return m


# ---------------------------------------------------- norms outside fp32 --

# one CTA a matrix (wide, tall), single SMs, CTA pairs
RANGE_SIZES = [(2, 40, 50), (2, 250, 120), (2, 140, 300), (2, 1000, 90), (40, 130, 300)]
EPS = float(torch.tensor(1e-30))  # the least that is taken, as the call sees it


def _scaled(m, exponent):
    return (m.to(D) * 10.0 ** exponent).to(FP)


@pytest.mark.parametrize("B,rows,cols", RANGE_SIZES)
@pytest.mark.parametrize("exponent", [-28, -24, -21, -17, 18, 22, 30, 39])
def test_newton_schulz_of_any_scale(moe, B, rows, cols, exponent):
    """Entries about 10^(exponent - 3): squares that vanish or overflow in fp32, and with
    39 a norm past fp32's largest number."""
    m = _scaled(_mats(B, rows, cols), exponent)
    m = m.clamp(-3e38, 3e38)
    want, norms = ref.newton_schulz(m, eps=EPS)
    _check_ns(_ns(moe, m, eps=EPS), want, _ns_bound(norms, 5), "fp32")
    mb = m.to(BF)
    want, norms = ref.newton_schulz(mb, eps=EPS)
    _check_ns(_ns(moe, mb, eps=EPS), want, _ns_bound(norms, 5), "bf16")


@pytest.mark.parametrize("B,rows,cols", RANGE_SIZES)
def test_newton_schulz_of_matrices_of_different_scales(moe, B, rows, cols):
    """One entry far above the others: its square is all that counts."""
    m = _mats(B, rows, cols)
    m[0] = _scaled(m[0], -20)
    m[0, rows // 2, cols // 3] = 1e-4
    m[1] = _scaled(m[1], 15)
    m[1, rows - 1, cols - 1] = 1e30
    want, norms = ref.newton_schulz(m, eps=EPS)
    _check_ns(_ns(moe, m, eps=EPS), want, _ns_bound(norms, 5), "spread")


@pytest.mark.parametrize("B,rows,cols", RANGE_SIZES)
@pytest.mark.parametrize("exponent,nesterov", [(-24, True), (-21, False), (22, True)])
def test_muon_step_of_any_scale(moe, B, rows, cols, exponent, nesterov):
    g = torch.Generator().manual_seed(rows)
    w = torch.randn(B, rows, cols, generator=g) * cols ** -0.5
    grad = _scaled(_mats(B, rows, cols, 7), exponent)
    lr, mu = 0.03, 0.5
    wt, vt = w.to(DEV), torch.zeros(B, rows, cols, device=DEV)
    ws = _ws(moe.newton_schulz_workspace_bytes(B, rows, cols))
    moe.muon_step(wt, None, vt, grad.to(DEV), torch.tensor([lr], device=DEV), mu, 0.0, 1.0, ws, nesterov=nesterov,
                  eps=EPS)
    assert moe.read_device_error(ws) == 0 and torch.equal(vt.cpu(), grad)
    o, norms = ref.newton_schulz(grad.to(D) * (1 + mu if nesterov else 1), eps=EPS)
    lr32 = float(torch.tensor(lr))
    err = (wt.cpu().to(D) - (w.to(D) - lr32 * o)).square().sum((1, 2)).sqrt()
    bound = lr32 * (_ns_bound(norms, 5) + 3 * 2.0 ** -24 * o.norm()) + 4 * 2.0 ** -24 * w.to(D).norm()
    assert bool((err <= bound).all()), float((err / bound).max())


@pytest.mark.parametrize("rows,cols", [(40, 50), (140, 300), (900, 1000)])
def test_newton_schulz_zero_and_non_finite_with_the_least_eps(moe, rows, cols):
    m = _scaled(_mats(5, rows, cols), -21)
    clean = _ns(moe, m, eps=EPS)
    m[1] = 0.0
    m[2, 3, 4] = float("nan")
    m[3, 0, 0] = float("inf")
    m[4] = float("nan")
    got = _ns(moe, m, eps=EPS)
    assert torch.equal(got[0], clean[0]) and not bool(got[1].any())
    for i in (2, 3, 4):
        assert bool(got[i].isnan().all())


def test_newton_schulz_norm_of_a_long_row(moe):
    """Equal values, whose fp32 sums err to one side: a chain of 4096 such additions is off
    by 6e-5.  With (1, 0, 0) the result is M / |M|: two roundings of the scaling, three of
    the norm, the pieces' 2^-22 and the product's two cuts of 2^-23 stay below 2^-19."""
    B, rows, cols = 620, 16, 65536  # so many matrices that a few CTAs sum one
    m = torch.full((B, rows, cols), 182 / 128, dtype=BF, device=DEV)
    out = torch.empty(B, rows, cols, device=DEV)
    ws = _ws(moe.newton_schulz_workspace_bytes(B, rows, cols))
    moe.newton_schulz(m, out, ws, steps=1, coefficients=(1.0, 0.0, 0.0))
    assert moe.read_device_error(ws) == 0
    want = (rows * cols) ** -0.5
    assert abs(float(out.min()) - want) <= 2.0 ** -19 * want and abs(float(out.max()) - want) <= 2.0 ** -19 * want
