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
