"""The dense operators' definitions in 64 bits (CPU torch), for the tests."""
import math

import torch

D = torch.float64
COEF = (3.4445, -4.7750, 2.0315)


def act(name, g):
    """act(g) and act'(g)."""
    if name == "relu":
        return g.clamp(min=0), (g > 0).to(g.dtype)
    z, dz = g, torch.ones_like(g)
    if name == "gelu":
        k = 2 * math.sqrt(2 / math.pi)
        z, dz = k * (g + 0.044715 * g ** 3), k * (1 + 3 * 0.044715 * g ** 2)
    s = torch.sigmoid(z)
    return g * s, s + g * s * (1 - s) * dz


def ffn(x, wg, wu, wd, add, scale, name):
    """y and what the backward needs, all unrounded."""
    x, wg, wu, wd = (t.to(D) for t in (x, wg, wu, wd))
    g, u = x @ wg.t(), x @ wu.t()
    a, da = act(name, g)
    h = a * u
    s = torch.ones(len(x), 1, dtype=D) if scale is None else scale.to(D)[:, None]
    y = s * (h @ wd.t())
    if add is not None:
        y = y + add.to(D)
    return dict(y=y, g=g, u=u, p=a, q=u * da, h=h, s=s)


def ffn_backward(f, x, wg, wu, wd, dy, dx_in):
    x, wg, wu, wd, dy = (t.to(D) for t in (x, wg, wu, wd, dy))
    r = dy @ wd
    du, dg = f["s"] * r * f["p"], f["s"] * r * f["q"]
    dx = dg @ wg + du @ wu
    if dx_in is not None:
        dx = dx + dx_in.to(D)
    return dict(r=r, du=du, dg=dg, dx=dx, dw_gate=dg.t() @ x, dw_up=du.t() @ x,
                dw_down=dy.t() @ (f["s"] * f["h"]), dscale=(r * f["h"]).sum(1))


def newton_schulz(m, steps=5, coef=None, eps=1e-7):
    """[B, rows, cols] in 64 bits, with the Frobenius norms of all iterates; coef: one
    triple a step."""
    m = m.to(D)
    tall = m.shape[1] > m.shape[2]
    x = m.transpose(1, 2) if tall else m
    x = x / (x.square().sum((1, 2), keepdim=True).sqrt() + eps)
    norms = [x.square().sum((1, 2)).sqrt()]
    for k in range(steps):
        a, b, c = COEF if coef is None else coef[k]
        s = x @ x.transpose(1, 2)
        x = a * x + (b * s + c * (s @ s)) @ x
        norms.append(x.square().sum((1, 2)).sqrt())
    return (x.transpose(1, 2) if tall else x), norms
