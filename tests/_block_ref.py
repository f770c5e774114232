"""The block operators' definitions in 64 bits (CPU torch), for the tests."""
import torch

D = torch.float64


def norm(s, gamma, beta, eps):
    """y, mean, rstd of rows s (already the stored sum)."""
    s = s.to(D)
    mean = s.mean(1)
    c = s - mean[:, None]
    rstd = 1 / torch.sqrt((c * c).mean(1) + eps)
    y = c * rstd[:, None]
    if gamma is not None:
        y = y * gamma.to(D)
    if beta is not None:
        y = y + beta.to(D)
    return y, mean, rstd


def norm_backward(s, dy, gamma, mean, rstd, dres):
    s, dy, mean, rstd = s.to(D), dy.to(D), mean.to(D)[:, None], rstd.to(D)[:, None]
    xh = (s - mean) * rstd
    w = dy if gamma is None else dy * gamma.to(D)
    dx = rstd * (w - w.mean(1, keepdim=True) - xh * (w * xh).mean(1, keepdim=True))
    if dres is not None:
        dx = dx + dres.to(D)
    return dx, (dy * xh).sum(0), dy.sum(0)


def balance(logits, idx, mask, N):
    """The forward's outputs; idx entries outside [0, N) are skipped."""
    T, K = idx.shape
    l = logits.to(D)
    live = torch.ones(T, dtype=torch.bool) if mask is None else mask != 0
    tc = int(live.sum())
    empty = (l == -float("inf")).all(1)
    use = live & ~empty
    lse, p = torch.zeros(T, dtype=D), torch.zeros(T, N, dtype=D)
    lse[live & empty] = -float("inf")
    if use.any():
        lse[use] = torch.logsumexp(l[use], 1)
        p[use] = torch.softmax(l[use], 1)
    flat = idx[live].reshape(-1).long()
    count = torch.bincount(flat[(flat >= 0) & (flat < N)], minlength=N)[:N]
    prob = p.sum(0) / max(tc, 1)
    f = count.to(D) / (max(tc, 1) * K)
    losses = torch.stack([N * (f * prob).sum(), (lse[use] ** 2).sum() / max(tc, 1)])
    return dict(expert_count=count, token_count=tc, expert_prob=prob, lse=lse, losses=losses)


def balance_backward(logits, idx, mask, count, tc, dlosses, dlogit):
    T, N = logits.shape
    K = idx.shape[1]
    l = logits.to(D)
    live = torch.ones(T, dtype=torch.bool) if mask is None else mask != 0
    use = live & ~(l == -float("inf")).all(1)
    out = torch.zeros(T, N, dtype=D)
    if tc > 0 and use.any():
        f = count.to(D) / (tc * K)
        p, lse = torch.softmax(l[use], 1), torch.logsumexp(l[use], 1)
        gb, gz = dlosses.to(D)
        out[use] = p * (gb * N / tc * (f - (p @ f)[:, None]) + gz * 2 / tc * lse[:, None])
    if dlogit is not None:
        for k in range(K):
            e = idx[:, k].long()
            ok = (e >= 0) & (e < N)
            out[ok, e[ok]] += dlogit[ok, k].to(D)
    return out


def mxint8(v):
    """Codes [rows, cols] and scale bytes [rows, cols / 32] of bf16 rows."""
    b = v.to(D).reshape(v.shape[0], v.shape[1] // 32, 32)
    m = b.abs().amax(2)
    bad = ~torch.isfinite(b).all(2)
    E = torch.where(m > 0, torch.frexp(torch.where(bad, 1.0, m))[1] - 1, -127).clamp(min=-127)
    step = ((E.to(torch.int64) - 6 + 1023) << 52).view(D)
    c = torch.round(torch.where(bad[:, :, None], 0.0, b) / step[:, :, None]).clamp(-127, 127)
    byte = torch.where(bad, 255, E + 127)
    return c.reshape(v.shape).to(torch.int8), byte.to(torch.uint8)


def mxint8_value(q, byte):
    e = byte.to(torch.int64)
    step = ((e - 133 + 1023) << 52).view(D)
    step = torch.where(e == 255, float("nan"), step)
    return q.to(D) * step.repeat_interleave(32, 1)
