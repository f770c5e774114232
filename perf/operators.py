"""The operators of a pre-norm training block around the routed-expert layer:
layer norm with the residual add, the router's balance loss with the dense
router gradient, and 8-bit activation checkpoints with their use in the
backward.  ``listed()`` and ``draw()`` give the cases, ``run()`` one pass in
plain torch (``own = False``) or through the library (``own = True``)."""
import math

import torch

own = False

DEV = "cuda"
EPS = 1e-5
BLOCK = 32  # elements that share one checkpoint scale


# ------------------------------------------------------------------ cases --

def listed():
    return [
        # one decoded token through the block's add + norm: latency only
        dict(name="norm_token", op="norm", T=1, d=2048, x="bf16", dy="fp32", add=True, affine=True, step=False),
        # the training step's norm at the OLMoE-like layer's shape
        dict(name="norm_olmoe", op="norm", T=8192, d=2048, x="bf16", dy="fp32", add=True, affine=True, step=True),
        # an fp32 residual stream, odd row count, a width that is no power of two
        dict(name="norm_odd_fp32", op="norm", T=1537, d=1000, x="fp32", dy="bf16", add=True, affine=True, step=True),
        # the wide layer's shape: the largest norm
        dict(name="norm_wide", op="norm", T=32768, d=4096, x="bf16", dy="fp32", add=True, affine=True, step=True),
        # the balance loss of the tiny layer: launch latency
        dict(name="balance_tiny", op="balance", T=256, N=8, K=2, mask=False, topk=True),
        # the fine-grained layer: 128 experts, skewed routing
        dict(name="balance_fine", op="balance", T=16384, N=128, K=8, mask=False, topk=True),
        # a long padded batch and an expert count that leaves rows unaligned
        dict(name="balance_long_padded", op="balance", T=131072, N=250, K=8, mask=True, topk=False),
        # the dense router gradient at the OLMoE-like and the wide layer's shapes
        dict(name="router_olmoe", op="router", T=8192, d=2048, N=64),
        dict(name="router_wide", op="router", T=32768, d=4096, N=32),
        # checkpoints of the tiny, the OLMoE-like and the fine-grained layer
        # (the last one with heavy drops: most of the buffer is tail)
        dict(name="checkpoint_tiny", op="checkpoint", T=256, d=128, N=8, K=2, h=256, cf=1.25, skew=0.0),
        dict(name="checkpoint_olmoe", op="checkpoint", T=8192, d=2048, N=64, K=8, h=1024, cf=1.25, skew=0.0),
        dict(name="checkpoint_fine", op="checkpoint", T=16384, d=2048, N=128, K=8, h=768, cf=1.0, skew=1.2),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["norm", "norm", "balance", "balance", "router", "checkpoint"])
    if op == "norm":
        T = _log_int(rng, 1, 32768)
        d = 8 * _log_int(rng, 8, max(8, min(1024, (12 << 20) // T)))
        return dict(op=op, T=T, d=d, x=rng.choice(["bf16", "fp32"]), dy=rng.choice(["bf16", "fp32"]),
                    add=rng.random() < 0.7, affine=rng.random() < 0.8, step=rng.random() < 0.7)
    if op == "balance":
        N = _log_int(rng, 2, 512)
        return dict(op=op, T=_log_int(rng, 1, min(131072, (1 << 25) // N)), N=N,
                    K=rng.randint(1, min(16, N)), mask=rng.random() < 0.5, topk=rng.random() < 0.5)
    if op == "router":
        T = _log_int(rng, 16, 32768)
        d = 8 * _log_int(rng, 8, 512)
        return dict(op=op, T=T, d=d, N=_log_int(rng, 2, max(2, min(512, (1 << 32) // (T * d)))))
    T = _log_int(rng, 16, 16384)
    N = _log_int(rng, 2, 128)
    d, h = 32 * _log_int(rng, 1, 64), 32 * _log_int(rng, 1, 32)
    return dict(op=op, T=T, d=d, N=N, K=rng.randint(1, min(8, N, max(1, (1 << 28) // (T * (d + 2 * h))))), h=h,
                cf=rng.choice([0.5, 1.0, 1.25, 2.0]), skew=rng.choice([0.0, 0.0, 0.6, 1.2]))


def _capacity(c):
    return math.ceil(c["cf"] * c["T"] * c["K"] / c["N"])


def _rows(c):
    return min(c["N"] * _capacity(c), c["T"] * c["K"])


def work(case):
    c = case

    def accepted():
        """Expected accepted routes: a token takes expert e with probability
        1 - exp(-z p_e) (K of N by popularity p), z such that these sum to K."""
        p = [(e + 1.0) ** -c["skew"] for e in range(c["N"])]
        p = [v / sum(p) for v in p]
        lo, hi = 0.0, 1e9
        for _ in range(200):
            z = 0.5 * (lo + hi)
            lo, hi = (z, hi) if sum(1 - math.exp(-z * v) for v in p) < c["K"] else (lo, z)
        take = [1 - math.exp(-lo * v) for v in p] if c["K"] < c["N"] else [1.0] * c["N"]
        return min(_rows(c), int(sum(min(c["T"] * q, _capacity(c)) for q in take)))

    if c["op"] == "norm":
        e = c["T"] * c["d"]
        xb, db = (2, 4)[c["x"] == "fp32"], (2, 4)[c["dy"] == "fp32"]
        nbytes = e * (xb + 2 + (2 + xb if c["add"] else 0)) + 8 * c["T"]
        if c["step"]:
            nbytes += e * (xb + db + 2 + 2)  # x, dy, the residual's gradient, dx
        return {"bytes": nbytes, "flops": e * (24 if c["step"] else 8)}
    if c["op"] == "balance":
        tn, tk = c["T"] * c["N"], c["T"] * c["K"]
        # the loss reads the logits, its gradient reads them again (it needs
        # every token's counts first) and writes as many
        return {"bytes": 12 * tn + 8 * tk + (4 * tk if c["topk"] else 0) + 8 * c["T"], "flops": 16 * tn}
    if c["op"] == "router":
        T, d, N = c["T"], c["d"], c["N"]
        return {"bytes": 10 * T * d + 4 * T * N + 8 * N * d, "flops": 4 * T * N * d}
    A, d, h = accepted(), c["d"], c["h"]
    save = 2 * A * (2 * h + d) + A * (2 * h + d) * 33 // 32
    restore = 2 * A * h * 33 // 32 + 6 * A * h
    back = 2 * c["T"] * d + A * d * 33 // 32 + 2 * A * d + 12 * c["T"] * c["K"]
    return {"bytes": save + restore + back, "flops": A * (3 * d + 12 * h)}


# ----------------------------------------------------------------- inputs --

def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(int(seed) * 7919 + 17)


def _normal(g, shape, std=1.0, dtype=torch.float32):
    return torch.randn(shape, generator=g, device=DEV).mul_(std).to(dtype)


def prepare(case, seed):
    c, g = case, _gen(seed)
    st = dict(case=dict(c), op=c["op"])
    if c["op"] == "norm":
        T, d = c["T"], c["d"]
        xt = torch.float32 if c["x"] == "fp32" else torch.bfloat16
        dt = torch.float32 if c["dy"] == "fp32" else torch.bfloat16
        # a residual stream: rows of different size, with an offset
        scale = torch.rand((T, 1), generator=g, device=DEV) * 2 + 0.5
        st["x"] = (_normal(g, (T, d)) * scale + 0.3).to(xt)
        st["add"] = _normal(g, (T, d), 0.5, torch.bfloat16) if c["add"] else None
        st["gamma"] = _normal(g, (d,), 0.1).add_(1.0) if c["affine"] else None
        st["beta"] = _normal(g, (d,), 0.1) if c["affine"] else None
        st["x_sum"] = torch.empty_like(st["x"]) if c["add"] else None
        st["y"] = torch.empty((T, d), dtype=torch.bfloat16, device=DEV)
        st["mean"] = torch.empty(T, device=DEV)
        st["rstd"] = torch.empty(T, device=DEV)
        if c["step"]:
            st["dy"] = _normal(g, (T, d), 1.0, dt)
            st["dres"] = _normal(g, (T, d), 1.0, torch.bfloat16)
            st["dx"] = torch.empty((T, d), dtype=torch.bfloat16, device=DEV)
            st["dgamma"] = torch.empty(d, device=DEV) if c["affine"] else None
            st["dbeta"] = torch.empty(d, device=DEV) if c["affine"] else None
    elif c["op"] == "balance":
        T, N, K = c["T"], c["N"], c["K"]
        # logits with a popularity offset per expert, as a router grows them
        st["logits"] = _normal(g, (T, N)).add_(_normal(g, (N,), 0.7))
        st["topk_idx"] = torch.topk(st["logits"], K, dim=1).indices.to(torch.int32)
        st["token_mask"] = None
        if c["mask"]:
            st["token_mask"] = (torch.rand(T, generator=g, device=DEV) < 0.85).to(torch.uint8)
        st["dlogit"] = _normal(g, (T, K), 0.01 / T) if c["topk"] else None
        st["dlosses"] = torch.tensor([0.01, 0.001], device=DEV)
        st["expert_count"] = torch.empty(N, dtype=torch.int32, device=DEV)
        st["token_count"] = torch.empty(1, dtype=torch.int32, device=DEV)
        st["expert_prob"] = torch.empty(N, device=DEV)
        st["lse"] = torch.empty(T, device=DEV)
        st["losses"] = torch.empty(2, device=DEV)
        st["dlogits"] = torch.empty((T, N), device=DEV)
    elif c["op"] == "router":
        T, d, N = c["T"], c["d"], c["N"]
        st["x"] = _normal(g, (T, d), 1.0, torch.bfloat16)
        st["w_router"] = _normal(g, (N, d), 0.02)
        # a few chosen logits carry most of a token's gradient
        big = torch.rand((T, N), generator=g, device=DEV) < 0.1
        st["dlogits"] = _normal(g, (T, N), 1e-2) * torch.where(big, 1.0, 0.05)
        st["dx_in"] = _normal(g, (T, d), 1e-3)
        st["dx"] = torch.empty((T, d), device=DEV)
        st["dw_router"] = torch.empty((N, d), device=DEV)
        st["dbias"] = torch.empty(N, device=DEV)
    else:
        T, d, N, K, h = (c[k] for k in ("T", "d", "N", "K", "h"))
        cap, R = _capacity(c), _rows(c)
        # routes: K distinct experts by popularity, slots in token order
        pop = -c["skew"] * torch.log(torch.arange(1, N + 1, device=DEV, dtype=torch.float32))
        u = torch.rand((T, N), generator=g, device=DEV).clamp_(1e-7, 1 - 1e-7)
        idx = torch.topk(pop - torch.log(-torch.log(u)), K, dim=1).indices
        hot = torch.zeros((T, N), dtype=torch.int32, device=DEV).scatter_(1, idx, 1)
        rank = (torch.cumsum(hot, 0) - hot).gather(1, idx)
        count = hot.sum(0).clamp(max=cap)
        offset = torch.zeros(N + 1, dtype=torch.int32, device=DEV)
        offset[1:] = torch.cumsum(count, 0)
        row = torch.where(rank < cap, offset[idx] + rank, torch.full_like(rank, -1))
        st["route_row"] = row.to(torch.int32).contiguous()
        st["expert_offset"] = offset
        st["topk_gate"] = torch.softmax(_normal(g, (T, K)), 1)
        # gate and up projections: some channels are much larger than others
        col = torch.exp(_normal(g, (1, h), 0.7))
        st["g_save"] = (_normal(g, (R, h)) * col).to(torch.bfloat16)
        st["u_save"] = _normal(g, (R, h), 1.0, torch.bfloat16)
        st["y_disp"] = _normal(g, (R, d), 0.5, torch.bfloat16)
        st["dy"] = _normal(g, (T, d), 1.0, torch.bfloat16)
        for n, cols in (("g", h), ("u", h), ("y", d)):
            st[n + "_q"] = torch.zeros((R, cols), dtype=torch.int8, device=DEV)
            st[n + "_scale"] = torch.zeros((R, cols // BLOCK), dtype=torch.uint8, device=DEV)
        # rows past the accepted ones are never written: they stay zero
        bf = dict(dtype=torch.bfloat16, device=DEV)
        st["g_out"], st["u_out"] = torch.zeros((R, h), **bf), torch.zeros((R, h), **bf)
        st["h_act"] = torch.zeros((R, h), **bf)
        st["dy_disp"] = torch.zeros((R, d), **bf)
        st["dgate"] = torch.empty((T, K), device=DEV)
    return st


# ------------------------------------------------------------------ plain --

def _plain_norm(st):
    s32 = st["x"].float()
    out = {}
    if st["add"] is not None:
        out["x_sum"] = (s32 + st["add"].float()).to(st["x"].dtype)
        s32 = out["x_sum"].float()
    mean = s32.mean(1, keepdim=True)
    xc = s32 - mean
    rstd = torch.rsqrt((xc * xc).mean(1, keepdim=True) + EPS)
    xh = xc * rstd
    y = xh if st["gamma"] is None else xh * st["gamma"] + st["beta"]
    out.update(y=y.to(torch.bfloat16), mean=mean[:, 0], rstd=rstd[:, 0])
    if not st["case"]["step"]:
        return out
    dy = st["dy"].float()
    w = dy if st["gamma"] is None else dy * st["gamma"]
    dx = rstd * (w - w.mean(1, keepdim=True) - xh * (w * xh).mean(1, keepdim=True)) + st["dres"].float()
    out["dx"] = dx.to(torch.bfloat16)
    if st["gamma"] is not None:
        out.update(dgamma=(dy * xh).sum(0), dbeta=dy.sum(0))
    return out


def _plain_balance(st):
    c = st["case"]
    T, N, K = c["T"], c["N"], c["K"]
    l, idx = st["logits"], st["topk_idx"].long()
    live = torch.ones(T, device=DEV) if st["token_mask"] is None else (st["token_mask"] != 0).float()
    tv = live.sum()
    inv = torch.where(tv > 0, 1.0 / tv.clamp(min=1.0), torch.zeros_like(tv))
    top = l.amax(1, keepdim=True)
    e = torch.exp(l - top)
    tot = e.sum(1, keepdim=True)
    p = e / tot * live[:, None]
    lse = (top + torch.log(tot))[:, 0] * live
    count = torch.zeros(N, device=DEV).index_add_(0, idx.reshape(-1), live[:, None].expand(T, K).reshape(-1))
    prob = p.sum(0) * inv
    f = count * inv / K
    losses = torch.stack([N * (f * prob).sum(), (lse * lse).sum() * inv])
    gb, gz = st["dlosses"][0], st["dlosses"][1]
    dl = p * (gb * N * inv * (f - (p * f).sum(1, keepdim=True)) + 2 * gz * inv * lse[:, None])
    if st["dlogit"] is not None:
        dl = dl.scatter_add(1, idx, st["dlogit"])
    return dict(expert_count=count.to(torch.int32), token_count=tv.to(torch.int32).reshape(1),
                expert_prob=prob, lse=lse, losses=losses, dlogits=dl)


def _plain_router(st):
    dl = st["dlogits"]
    return dict(dx=st["dx_in"] + dl @ st["w_router"], dw_router=dl.t() @ st["x"].float(), dbias=dl.sum(0))


def _plain_mxint8(v):
    """Codes and scales of [R, cols] values, in blocks of 32 along a row."""
    b = v.float().reshape(v.shape[0], -1, BLOCK)
    bits = b.abs().amax(2).view(torch.int32)
    byte = bits >> 23  # the exponent of the block's largest magnitude, + 127
    inv = ((254 - byte.clamp(max=254)) << 23).view(torch.float32)  # 2^-E
    inv = torch.where(byte >= 254, torch.full_like(inv, 2.0 ** -127), inv)
    code = torch.round(b * inv[:, :, None] * 64).clamp(-127, 127).to(torch.int8)
    return code, byte.to(torch.uint8)


def _plain_value(code, byte):
    e = byte.to(torch.int32)
    scale = torch.where(e == 0, 1 << 22, e << 23).view(torch.float32)  # 2^(byte - 127)
    scale = torch.where(e == 255, float("nan"), scale)
    return (code.float() / 64 * scale[:, :, None]).reshape(code.shape[0], -1)


def _plain_checkpoint(st):
    R = st["g_save"].shape[0]
    live = (torch.arange(R, device=DEV) < st["expert_offset"][-1])[:, None]
    g, u, y = (_plain_value(*_plain_mxint8(st[n])) for n in ("g_save", "u_save", "y_disp"))
    g, u = g * live, u * live
    h = g / (1 + torch.exp(-g)) * u
    row = st["route_row"].long()
    on = row >= 0
    dy, gate = st["dy"].float(), st["topk_gate"]
    dgate = (y[row.clamp(min=0)] * dy[:, None, :]).sum(2) * on
    dy_disp = torch.zeros_like(st["dy_disp"])
    t, k = torch.nonzero(on, as_tuple=True)
    dy_disp[row[t, k]] = (gate[t, k][:, None] * dy[t]).to(torch.bfloat16)
    bf = torch.bfloat16
    return dict(g=g.to(bf), u=u.to(bf), h=h.to(bf), dy_disp=dy_disp, dgate=dgate)


# -------------------------------------------------------------------- own --

def _own_norm(st, moe):
    c = st["case"]
    moe.layer_norm(st["x"], st["add"], st["gamma"], st["beta"], EPS, st["x_sum"], st["y"], st["mean"], st["rstd"])
    out = dict(y=st["y"], mean=st["mean"], rstd=st["rstd"])
    if c["add"]:
        out["x_sum"] = st["x_sum"]
    if not c["step"]:
        return out
    if "ws" not in st:
        st["ws"] = torch.zeros(moe.layer_norm_backward_workspace_bytes(c["T"], c["d"]), dtype=torch.uint8, device=DEV)
    moe.layer_norm_backward(st["x_sum"] if c["add"] else st["x"], st["dy"], st["gamma"], st["mean"], st["rstd"],
                            st["dres"], st["dx"], st["dgamma"], st["dbeta"], st["ws"])
    out["dx"] = st["dx"]
    if c["affine"]:
        out.update(dgamma=st["dgamma"], dbeta=st["dbeta"])
    return out


def _own_balance(st, moe):
    if "ws" not in st:
        c = st["case"]
        st["shape"] = moe.Shape(c["T"], 8, c["N"], c["K"], 8, 1)
        st["ws"] = torch.zeros(moe.balance_loss_workspace_bytes(st["shape"]), dtype=torch.uint8, device=DEV)
    s = st["shape"]
    moe.balance_loss(s, st["logits"], st["topk_idx"], st["token_mask"], st["expert_count"], st["token_count"],
                     st["expert_prob"], st["lse"], st["losses"], st["ws"])
    moe.balance_loss_backward(s, st["logits"], st["topk_idx"], st["token_mask"], st["expert_count"],
                              st["token_count"], st["lse"], st["dlosses"], st["dlogit"], st["dlogits"])
    return {n: st[n] for n in ("expert_count", "token_count", "expert_prob", "lse", "losses", "dlogits")}


def _own_router(st, moe):
    if "ws" not in st:
        c = st["case"]
        st["shape"] = moe.Shape(c["T"], c["d"], c["N"], 1, 8, 1)
        st["ws"] = torch.zeros(moe.router_dense_backward_workspace_bytes(st["shape"]), dtype=torch.uint8, device=DEV)
    moe.router_dense_backward(st["shape"], st["x"], st["w_router"], st["dlogits"], st["dx_in"], st["dx"],
                              st["dw_router"], st["dbias"], st["ws"])
    return {n: st[n] for n in ("dx", "dw_router", "dbias")}


def _own_checkpoint(st, moe):
    if "shape" not in st:
        c = st["case"]
        st["shape"] = moe.Shape(c["T"], c["d"], c["N"], c["K"], c["h"], _capacity(c))
    s, off = st["shape"], st["expert_offset"]
    moe.checkpoint_save(s, off, st["g_save"], st["u_save"], st["y_disp"], st["g_q"], st["g_scale"], st["u_q"],
                        st["u_scale"], st["y_q"], st["y_scale"])
    moe.combine_backward_checkpoint(s, st["dy"], st["y_q"], st["y_scale"], st["route_row"], st["topk_gate"],
                                    st["dy_disp"], st["dgate"])
    moe.checkpoint_restore(s, off, st["g_q"], st["g_scale"], st["u_q"], st["u_scale"], st["g_out"], st["u_out"],
                           st["h_act"])
    return dict(g=st["g_out"], u=st["u_out"], h=st["h_act"], dy_disp=st["dy_disp"], dgate=st["dgate"])


_PLAIN = dict(norm=_plain_norm, balance=_plain_balance, router=_plain_router, checkpoint=_plain_checkpoint)
_OWN = dict(norm=_own_norm, balance=_own_balance, router=_own_router, checkpoint=_own_checkpoint)


def run(state):
    if own:
        import combine_expert_gemm_gb300 as moe
        return _OWN[state["op"]](state, moe)
    return _PLAIN[state["op"]](state)


# ------------------------------------------------------------------ exact --

def exact(case, seed):
    """run()'s outputs from the definitions in 64 bits."""
    st, D = prepare(case, seed), torch.float64
    T = case["T"]
    if case["op"] == "norm":
        d, s, out = case["d"], st["x"].to(D), {}
        if case["add"]:
            # the stored sum is what is normalised: its rounding is part of the definition
            s = (s + st["add"].to(D)).to(st["x"].dtype).to(D)
            out["x_sum"] = s
        var, mean = torch.var_mean(s, dim=1, correction=0)
        rstd = (var + EPS) ** -0.5
        one = torch.ones(d, dtype=D, device=DEV)
        gamma = one if st["gamma"] is None else st["gamma"].to(D)
        xh = torch.addcmul(-(mean * rstd)[:, None], s, rstd[:, None])
        out.update(mean=mean, rstd=rstd, y=xh * gamma + (0 if st["beta"] is None else st["beta"].to(D)))
        if case["step"]:
            dy = st["dy"].to(D)
            a = torch.mv(dy, gamma) / d
            b = torch.mv(dy * xh, gamma) / d
            out["dx"] = st["dres"].to(D) + rstd[:, None] * (dy * gamma - a[:, None] - b[:, None] * xh)
            if case["affine"]:
                out["dgamma"] = torch.einsum("td,td->d", dy, xh)
                out["dbeta"] = torch.einsum("td->d", dy)
        return out
    if case["op"] == "balance":
        N, K = case["N"], case["K"]
        keep = torch.arange(T, device=DEV) if st["token_mask"] is None else torch.nonzero(st["token_mask"])[:, 0]
        tv = len(keep)
        l, idx = st["logits"].to(D)[keep], st["topk_idx"].long()
        lse = torch.logsumexp(l, 1)
        p = torch.softmax(l, 1)
        count = torch.bincount(idx[keep].reshape(-1), minlength=N)
        prob, f = (p.mean(0), count / (tv * K)) if tv else (p.sum(0), count.to(D))
        gb, gz = st["dlosses"].to(D)
        losses = torch.stack([N * torch.dot(f.to(D), prob), lse.square().sum() / max(tv, 1)])
        dlogits = torch.zeros((T, N), dtype=D, device=DEV)
        if tv:
            up = (gb * N / tv) * f.to(D)  # d balance / d p, for each expert
            dlogits[keep] = p * (up - (p @ up)[:, None] + (2 * gz / tv) * lse[:, None])
        if st["dlogit"] is not None:
            for k in range(K):
                dlogits[torch.arange(T, device=DEV), idx[:, k]] += st["dlogit"][:, k].to(D)
        full = torch.zeros(T, dtype=D, device=DEV)
        full[keep] = lse
        return dict(expert_count=None, token_count=None, expert_prob=prob, lse=full, losses=losses, dlogits=dlogits)
    if case["op"] == "router":
        dl, x, w = st["dlogits"].to(D), st["x"].to(D), st["w_router"].to(D)
        return dict(dx=torch.addmm(st["dx_in"].to(D), dl, w), dw_router=torch.einsum("tn,td->nd", dl, x),
                    dbias=torch.einsum("tn->n", dl))
    A = int(st["expert_offset"][-1])

    def held(v):
        """The value that the 8-bit checkpoint of v holds."""
        b = v[:A].to(D).reshape(-1, BLOCK)
        E = (torch.frexp(b.abs().amax(1))[1] - 1).clamp(min=-127)
        step = ((E.to(torch.int64) - 6 + 1023) << 52).view(D)[:, None]  # 2^(E - 6)
        q = torch.round(b / step).clamp(-127, 127) * step
        out = torch.zeros(v.shape, dtype=D, device=DEV)
        out[:A] = q.reshape(A, -1)
        return out

    g, u, y = held(st["g_save"]), held(st["u_save"]), held(st["y_disp"])
    dy, gate, row = st["dy"].to(D), st["topk_gate"].to(D), st["route_row"].long()
    dgate = torch.zeros(row.shape, dtype=D, device=DEV)
    dy_disp = torch.zeros(st["dy_disp"].shape, dtype=D, device=DEV)
    for k in range(case["K"]):
        t = torch.nonzero(row[:, k] >= 0)[:, 0]
        r = row[t, k]
        dgate[t, k] = torch.einsum("rd,rd->r", dy[t], y[r])
        dy_disp[r] = gate[t, k][:, None] * dy[t]
    return dict(g=g, u=u, h=g * torch.sigmoid(g) * u, dy_disp=dy_disp, dgate=dgate)
