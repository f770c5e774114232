"""Long sums of the gated feed-forward backward.  The tensor core cuts an fp32 sum by
up to 2^-23 of its size where it adds 16 products, always towards zero, so sums of terms
of one sign show what a long one loses.  The factors that the tensor cores multiply
are exact here or taken from the call itself, which leaves the sum's own error: at
most 512 cuts in one accumulator, then additions that round to nearest."""
import pytest
import torch

from _gpu_util import DEV
from test_gpu_dense import _ws

pytestmark = pytest.mark.gpu
BF, D = torch.bfloat16, torch.float64
CUTS = 512  # of one accumulator


@pytest.fixture(scope="module")
def moe():
    import __graft_entry__
    __graft_entry__.build()
    import combine_expert_gemm_gb300 as m
    return m


def _positive(g, *s):
    return (1 + torch.rand(*s, generator=g)).to(BF).to(DEV)


def _step(moe, x, wg, wu, wd, dy, dw_type=torch.float32, scale=None):
    (T, d), h = x.shape, wg.shape[0]
    ws = _ws(max(moe.gated_ffn_workspace_bytes(T, d, h), moe.gated_ffn_backward_workspace_bytes(T, d, h)))
    y = torch.empty_like(x)
    hb, p, q = (torch.empty(T, h, dtype=BF, device=DEV) for _ in range(3))
    moe.gated_ffn(x, wg, wu, wd, None, scale, y, hb, p, q, ws, act="relu")
    dx = torch.empty(T, d, device=DEV)
    dw = [torch.empty(s, dtype=dw_type, device=DEV) for s in ((h, d), (h, d), (d, h))]
    moe.gated_ffn_backward(x, wg, wu, wd, scale, hb, p, q, dy, None, dx, *dw, None, ws)
    assert moe.read_device_error(ws) == 0
    return hb, p, q, dx, dw


def _close(got, want, terms, what):
    """terms: of the sum, all of one sign; its accumulators are added in fp32."""
    cuts = min(CUTS, -(-terms // 16))
    tol = cuts * 2.0 ** -23 + (-(-terms // (16 * CUTS)) + 1) * 2.0 ** -24 + torch.finfo(got.dtype).eps / 2
    off = float(((got.cpu().to(D) - want) / want).abs().max())
    assert off <= tol, f"{what}: {off:.3g}, {tol:.3g} allowed"


@pytest.mark.parametrize("T,d,h", [(2000, 72, 40), (8192, 8, 8), (30001, 264, 136), (1 << 20, 8, 8)])
@pytest.mark.parametrize("dw_type", [torch.float32, BF])
def test_weight_gradients_of_many_tokens(moe, T, d, h, dw_type):
    g = torch.Generator().manual_seed(T + d)
    x, dy = _positive(g, T, d), _positive(g, T, d)
    wg, wu = _positive(g, h, d) / d, _positive(g, h, d) / d
    wd = torch.zeros(d, h, dtype=BF, device=DEV)
    wd[torch.arange(h) % d, torch.arange(h)] = 1.0  # each hidden unit has one output, so R is dy's value
    hb, p, q, dx, dw = _step(moe, x, wg, wu, wd, dy, dw_type)
    r = dy[:, torch.arange(h) % d].float()
    du, dg = (r * p.float()).to(BF), (r * q.float()).to(BF)
    c = lambda t: t.cpu().to(D)
    _close(dw[0], c(dg).t() @ c(x), T, "dw_gate")
    _close(dw[1], c(du).t() @ c(x), T, "dw_up")
    _close(dw[2], c(dy).t() @ c(hb), T, "dw_down")


@pytest.mark.parametrize("T,d,h", [(300, 72, 65536), (64, 8, 20000), (700, 264, 8200)])
def test_input_gradient_of_many_hidden_units(moe, T, d, h):
    g = torch.Generator().manual_seed(T + d)
    x, dy = _positive(g, T, d), _positive(g, T, d)
    wg, wu = _positive(g, h, d) / d, _positive(g, h, d) / d
    wd = torch.zeros(d, h, dtype=BF, device=DEV)
    wd[torch.arange(h) % d, torch.arange(h)] = 1.0
    hb, p, q, dx, dw = _step(moe, x, wg, wu, wd, dy)
    r = dy[:, torch.arange(h) % d].float()
    c = lambda t: t.cpu().to(D)
    want = c((r * q.float()).to(BF)) @ c(wg) + c((r * p.float()).to(BF)) @ c(wu)
    _close(dx, want, 2 * h, "dx")


def test_input_and_weight_gradients_of_the_offset_test(moe):
    """More than 2^31 elements of x and dy; the weights' gradients of all of them."""
    T, d, h = 1050001, 2056, 8
    g = torch.Generator(device=DEV).manual_seed(1)
    x = torch.rand(T, d, generator=g, device=DEV, dtype=BF).add_(1)
    dy = torch.rand(T, d, generator=g, device=DEV, dtype=BF).add_(1)
    wg, wu = (torch.rand(h, d, generator=g, device=DEV).add_(1).div_(d).to(BF) for _ in range(2))
    wd = torch.zeros(d, h, dtype=BF, device=DEV)
    wd[torch.arange(h), torch.arange(h)] = 1.0
    hb, p, q, dx, dw = _step(moe, x, wg, wu, wd, dy)
    r = dy[:, :h].float()
    du, dg = (r * p.float()).to(BF), (r * q.float()).to(BF)
    want = [torch.zeros(s, dtype=D) for s in ((h, d), (h, d), (d, h))]
    for i in range(0, T, 100000):
        c = lambda t: t[i:i + 100000].cpu().to(D)
        xs, ys = c(x), c(dy)
        want[0] += c(dg).t() @ xs
        want[1] += c(du).t() @ xs
        want[2] += ys.t() @ c(hb)
    for name, a, b in zip(("dw_gate", "dw_up", "dw_down"), dw, want):
        _close(a, b, T, name)
