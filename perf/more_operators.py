"""A shared expert beside the routed ones and the update of the weight matrices:
the dense gated feed-forward block, forward alone and with its backward, the
Newton-Schulz orthogonalisation of batches of matrices and the Muon step built
on it.  ``listed()`` and ``draw()`` give the cases, ``run()`` one pass in plain
torch (``own = False``) or through the library (``own = True``)."""
import math

import torch

own = False

DEV = "cuda"
EPS = 1e-7
STEPS = 5
COEF = (3.4445, -4.7750, 2.0315)  # the quintic that lifts small singular values fastest
MOST_FFN = 32768 * 4096 * 2048    # T d h of the largest feed-forward case


# ------------------------------------------------------------------ cases --

def listed():
    return [
        # one decoded token through a shared expert of the OLMoE-like width: latency only
        dict(name="ffn_token", op="ffn", T=1, d=2048, h=1024, act="silu", add=True, scale=False, step=False),
        # a decoded batch through the wide layer's shared expert, gated per token
        dict(name="ffn_batch", op="ffn", T=96, d=4096, h=2048, act="silu", add=True, scale=True, step=False),
        # a ragged prompt, widths that no tile divides
        dict(name="ffn_odd", op="ffn", T=1537, d=1000, h=712, act="gelu", add=True, scale=False, step=False),
        # the wide layer's batch: the largest forward
        dict(name="ffn_wide", op="ffn", T=32768, d=4096, h=2048, act="silu", add=True, scale=False, step=False),
        # training steps: forward with saving and backward, at the OLMoE-like layer's shape
        dict(name="step_olmoe", op="ffn", T=8192, d=2048, h=1024, act="silu", add=True, scale=False, step=True),
        # a short ragged batch with a token gate and its gradient
        dict(name="step_odd", op="ffn", T=777, d=1000, h=1416, act="gelu", add=True, scale=True, step=True),
        # the orthogonal factor alone: a few ragged matrices, and one matrix of a wide shared expert
        dict(name="ns_odd", op="ns", B=3, rows=1001, cols=717, dtype="bf16"),
        dict(name="ns_shared", op="ns", B=1, rows=2048, cols=4096, dtype="fp32"),
        # the experts of the tiny layer: launch latency
        dict(name="muon_tiny", op="muon", B=8, rows=256, cols=128, nesterov=True, copy=True),
        # the down projections of the fine-grained layer: more rows than columns
        dict(name="muon_fine_down", op="muon", B=128, rows=2048, cols=768, nesterov=True, copy=True),
        # the gate projections of the OLMoE-like layer: the largest update
        dict(name="muon_olmoe", op="muon", B=64, rows=1024, cols=2048, nesterov=True, copy=True),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _ns_flops(c):
    m, n = min(c["rows"], c["cols"]), max(c["rows"], c["cols"])
    return c["B"] * STEPS * (4 * m * m * n + 2 * m * m * m)


def draw(rng):
    op = rng.choice(["ffn", "ffn", "step", "ns", "muon", "muon"])
    if op in ("ffn", "step"):
        d, h = 8 * _log_int(rng, 8, 512), 8 * _log_int(rng, 8, 512)
        most = min(32768, MOST_FFN // (d * h) // (3 if op == "step" else 1))
        return dict(op="ffn", T=_log_int(rng, 1, most), d=d, h=h, act=rng.choice(["silu", "silu", "gelu", "relu"]),
                    add=rng.random() < 0.7, scale=rng.random() < 0.4, step=op == "step")
    c = dict(op=op, B=1, rows=_log_int(rng, 16, 4096), cols=_log_int(rng, 16, 4096))
    c["B"] = _log_int(rng, 1, max(1, min(128, (1 << 27) // (c["rows"] * c["cols"]), int(3.4e12 / _ns_flops(c)))))
    if op == "ns":
        return dict(c, dtype=rng.choice(["bf16", "fp32"]))
    return dict(c, nesterov=rng.random() < 0.7, copy=rng.random() < 0.8)


def work(case):
    c = case
    if c["op"] == "ffn":
        T, d, h = c["T"], c["d"], c["h"]
        nbytes = 2 * T * d * (3 if c["add"] else 2) + 6 * d * h + 2 * T * h + (4 * T if c["scale"] else 0)
        if c["step"]:
            # the saved factors are written and read, the weights and x read again,
            # dy read, dx and the weights' gradients written
            nbytes += 2 * (4 * T * h) + 2 * T * h + 6 * d * h + 2 * T * d * 3 + 6 * d * h
            nbytes += 8 * T if c["scale"] else 0
        return {"bytes": nbytes, "flops": (18 if c["step"] else 6) * T * d * h}
    e = c["B"] * c["rows"] * c["cols"]
    if c["op"] == "ns":
        return {"bytes": e * (4 if c["dtype"] == "bf16" else 8), "flops": _ns_flops(c)}
    return {"bytes": e * (22 if c["copy"] else 20), "flops": _ns_flops(c) + 8 * e}


# ----------------------------------------------------------------- inputs --

def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(int(seed) * 7919 + 29)


def _normal(g, shape, std=1.0, dtype=torch.float32):
    return torch.randn(shape, generator=g, device=DEV).mul_(std).to(dtype)


def _matrices(g, B, rows, cols, std):
    """Gradients of weight matrices: a few strong directions over a floor of noise."""
    r = max(1, min(rows, cols) // 8)
    left = torch.randn((B, rows, r), generator=g, device=DEV)
    left *= torch.exp(-3.0 * torch.arange(r, device=DEV) / r)
    right = torch.randn((B, r, cols), generator=g, device=DEV)
    return (left @ right).mul_(r ** -0.5).add_(torch.randn((B, rows, cols), generator=g, device=DEV), alpha=0.3).mul_(std)


def prepare(case, seed):
    c, g = case, _gen(seed)
    st = dict(case=dict(c), op=c["op"])
    bf = dict(dtype=torch.bfloat16, device=DEV)
    if c["op"] == "ffn":
        T, d, h = c["T"], c["d"], c["h"]
        st["x"] = _normal(g, (T, d), 1.0, torch.bfloat16)  # rows of a layer norm
        st["w_gate"] = _normal(g, (h, d), d ** -0.5, torch.bfloat16)
        st["w_up"] = _normal(g, (h, d), d ** -0.5, torch.bfloat16)
        st["w_down"] = _normal(g, (d, h), h ** -0.5, torch.bfloat16)
        st["add"] = _normal(g, (T, d), 0.5, torch.bfloat16) if c["add"] else None
        st["scale"] = torch.sigmoid(_normal(g, (T,))) if c["scale"] else None
        st["y"], st["h_act"] = torch.empty((T, d), **bf), torch.empty((T, h), **bf)
        if c["step"]:
            st["p"], st["q"] = torch.empty((T, h), **bf), torch.empty((T, h), **bf)
            st["dy"] = _normal(g, (T, d), 1.0, torch.bfloat16)
            st["dx_in"] = _normal(g, (T, d), 0.5, torch.bfloat16)
            st["dx"] = torch.empty((T, d), **bf)
            st["dw_gate"], st["dw_up"] = torch.empty((h, d), **bf), torch.empty((h, d), **bf)
            st["dw_down"] = torch.empty((d, h), **bf)
            st["dscale"] = torch.empty(T, **bf) if c["scale"] else None
        return st
    B, rows, cols = c["B"], c["rows"], c["cols"]
    if c["op"] == "ns":
        dt = torch.bfloat16 if c["dtype"] == "bf16" else torch.float32
        st["m"] = _matrices(g, B, rows, cols, 1e-3).to(dt)
        st["out"] = torch.empty_like(st["m"])
        return st
    st["grad"] = _matrices(g, B, rows, cols, 1e-3)
    st["momentum"] = _matrices(g, B, rows, cols, 5e-3)
    st["w"] = _normal(g, (B, rows, cols), cols ** -0.5)
    st["w_copy"] = st["w"].to(torch.bfloat16) if c["copy"] else None
    st["lr"] = torch.tensor([0.02], device=DEV)
    st["mu"], st["decay"], st["factor"] = 0.95, 0.01, max(1.0, rows / cols) ** 0.5
    return st


# ------------------------------------------------------------------ plain --

def _plain_act(act, g):
    """act(g) and its derivative."""
    if act == "relu":
        on = (g > 0).float()
        return g * on, on
    z, dz = g, 1.0
    if act == "gelu":
        k = 2 * math.sqrt(2 / math.pi)
        z, dz = k * (g + 0.044715 * g * g * g), k * (1 + 3 * 0.044715 * g * g)
    s = 1 / (1 + torch.exp(-z))
    return g * s, s + g * s * (1 - s) * dz


def _plain_ffn(st):
    c, bf = st["case"], torch.bfloat16
    x, wg, wu, wd = (st[n].float() for n in ("x", "w_gate", "w_up", "w_down"))
    g, u = x @ wg.t(), x @ wu.t()
    a, da = _plain_act(c["act"], g)
    h = a * u
    y = h @ wd.t()
    scale = None if st["scale"] is None else st["scale"][:, None]
    if scale is not None:
        y = y * scale
    if st["add"] is not None:
        y = y + st["add"].float()
    out = dict(y=y.to(bf))
    if not c["step"]:
        return out
    dy = st["dy"].float()
    dhr = dy @ wd
    sh, dh = h, dhr
    if scale is not None:
        out["dscale"] = (dhr * h).sum(1).to(bf)
        sh, dh = h * scale, dhr * scale
    dg, du = dh * u * da, dh * a
    out["dx"] = (st["dx_in"].float() + dg @ wg + du @ wu).to(bf)
    out.update(dw_gate=(dg.t() @ x).to(bf), dw_up=(du.t() @ x).to(bf), dw_down=(dy.t() @ sh).to(bf))
    return out


def _plain_ns(m):
    """The Newton-Schulz factor of [B, rows, cols] fp32 matrices."""
    tall = m.shape[1] > m.shape[2]
    x = m.transpose(1, 2) if tall else m
    x = x / (x.square().sum((1, 2), keepdim=True).sqrt() + EPS)
    a, b, c = COEF
    for _ in range(STEPS):
        s = x @ x.transpose(1, 2)
        x = a * x + (b * s + c * (s @ s)) @ x
    return x.transpose(1, 2) if tall else x


def _plain_muon(st):
    mu, v, w = st["mu"], st["momentum"], st["w"]
    v.mul_(mu).add_(st["grad"])
    o = _plain_ns(st["grad"] + mu * v if st["case"]["nesterov"] else v)
    w.mul_(1 - st["lr"] * st["decay"]).sub_(st["lr"] * st["factor"] * o)
    out = dict(w=w, momentum=v)
    if st["w_copy"] is not None:
        st["w_copy"].copy_(w)
        out["w_copy"] = st["w_copy"]
    return out


# -------------------------------------------------------------------- own --

def _ws(n):
    ws = torch.empty(n, dtype=torch.uint8, device=DEV)
    ws[:256] = 0  # the status word
    return ws


def _own_ffn(st, moe):
    c = st["case"]
    T, d, h = c["T"], c["d"], c["h"]
    if "ws" not in st:
        n = moe.gated_ffn_workspace_bytes(T, d, h)
        st["ws"] = _ws(max(n, moe.gated_ffn_backward_workspace_bytes(T, d, h)) if c["step"] else n)
    w = (st["w_gate"], st["w_up"], st["w_down"])
    moe.gated_ffn(st["x"], *w, st["add"], st["scale"], st["y"], st["h_act"], st.get("p"), st.get("q"), st["ws"],
                  act=c["act"])
    if not c["step"]:
        return dict(y=st["y"])
    moe.gated_ffn_backward(st["x"], *w, st["scale"], st["h_act"], st["p"], st["q"], st["dy"], st["dx_in"], st["dx"],
                           st["dw_gate"], st["dw_up"], st["dw_down"], st["dscale"], st["ws"])
    return {n: st[n] for n in ("y", "dx", "dw_gate", "dw_up", "dw_down", "dscale") if st[n] is not None}


def _own_ns(st, moe):
    c = st["case"]
    if "ws" not in st:
        st["ws"] = _ws(moe.newton_schulz_workspace_bytes(c["B"], c["rows"], c["cols"]))
    moe.newton_schulz(st["m"], st["out"], st["ws"], eps=EPS)
    return dict(out=st["out"])


def _own_muon(st, moe):
    c = st["case"]
    if "ws" not in st:
        st["ws"] = _ws(moe.newton_schulz_workspace_bytes(c["B"], c["rows"], c["cols"]))
    moe.muon_step(st["w"], st["w_copy"], st["momentum"], st["grad"], st["lr"], st["mu"], st["decay"], st["factor"],
                  st["ws"], nesterov=c["nesterov"], eps=EPS)
    out = dict(w=st["w"], momentum=st["momentum"])
    if c["copy"]:
        out["w_copy"] = st["w_copy"]
    return out


def run(state):
    if own:
        import combine_expert_gemm_gb300 as moe
        return dict(ffn=_own_ffn, ns=_own_ns, muon=_own_muon)[state["op"]](state, moe)
    if state["op"] == "ffn":
        return _plain_ffn(state)
    if state["op"] == "ns":
        return dict(out=_plain_ns(state["m"].float()).to(state["m"].dtype))
    return _plain_muon(state)


# ------------------------------------------------------------------ exact --

def _exact_ns(m):
    """Each matrix by its Gram matrix's polynomial: with S = X X^T of the short
    side, X_k = p_k(S) X and the factors p_k(S) commute with S."""
    small_rows = m.shape[-2] <= m.shape[-1]
    out = torch.empty_like(m)
    for i in range(m.shape[0]):
        x = m[i] if small_rows else m[i].mT
        x = x / (torch.linalg.vector_norm(x) + EPS)
        for _ in range(STEPS):
            gram = torch.einsum("in,jn->ij", x, x)
            poly = torch.addmm(gram * COEF[1], gram, gram, alpha=COEF[2])
            poly.diagonal().add_(COEF[0])
            x = torch.mm(poly, x)
        out[i] = x if small_rows else x.mT
    return out


def exact(case, seed):
    """run()'s outputs from the definitions in 64 bits."""
    st, D = prepare(case, seed), torch.float64
    if case["op"] == "ns":
        return dict(out=_exact_ns(st["m"].to(D)))
    if case["op"] == "muon":
        g, mu, lr = st["grad"].to(D), st["mu"], float(st["lr"])
        v = torch.add(g, st["momentum"].to(D), alpha=mu)
        o = _exact_ns(torch.add(g, v, alpha=mu) if case["nesterov"] else v)
        w = st["w"].to(D) * (1 - lr * st["decay"]) - lr * st["factor"] * o
        out = dict(w=w, momentum=v)
        if case["copy"]:
            out["w_copy"] = w
        return out
    # the block's derivatives by reverse accumulation over 64-bit operations
    leaf = {n: st[n].to(D).requires_grad_(case["step"]) for n in ("x", "w_gate", "w_up", "w_down")}
    s = torch.ones(case["T"], dtype=D, device=DEV) if st["scale"] is None else st["scale"].to(D)
    s.requires_grad_(case["step"])
    F = torch.nn.functional
    act = dict(silu=F.silu, gelu=lambda v: F.gelu(v, approximate="tanh"), relu=F.relu)[case["act"]]
    hidden = act(F.linear(leaf["x"], leaf["w_gate"])) * F.linear(leaf["x"], leaf["w_up"])
    y = F.linear(hidden, leaf["w_down"]) * s[:, None]
    out = dict(y=(y if st["add"] is None else y + st["add"].to(D)).detach())
    if case["step"]:
        names = ("x", "w_gate", "w_up", "w_down")
        grads = torch.autograd.grad(y, [leaf[n] for n in names] + [s], st["dy"].to(D))
        out.update(dx=grads[0] + st["dx_in"].to(D), dw_gate=grads[1], dw_up=grads[2], dw_down=grads[3])
        if case["scale"]:
            out["dscale"] = grads[4]
    return out
