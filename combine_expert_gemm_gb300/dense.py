"""Python binding of the dense operators beside the routed experts
(``include/moe_dense.h``): the gated feed-forward block of a shared expert, and
the Newton-Schulz orthogonalisation with the Muon step that updates weight
matrices.

Argument marshalling only, as in the package's ``__init__``.  Weights, their gradients
and the matrices of Newton-Schulz and Muon have exactly the shape that the call
states (a transposed one has as many elements); of the tokens' buffers, which may go on
behind the last row, the number of elements is compared, as in a training block.
"""
import ctypes

import torch

from . import _P, _SZ, _bf16, _check, _f32, _lib
from .block import _DTYPE, _arg, _float_type, _keep, _on, _ws

__all__ = ["gated_ffn", "gated_ffn_workspace_bytes", "gated_ffn_backward",
           "gated_ffn_backward_workspace_bytes", "newton_schulz", "newton_schulz_workspace_bytes",
           "muon_step", "SharedExpert", "Muon"]

_I, _F = ctypes.c_int32, ctypes.c_float
_SIG = {
    "moe_gated_ffn_workspace_bytes": ([_I] * 3, _SZ),
    "moe_gated_ffn_backward_workspace_bytes": ([_I] * 3, _SZ),
    "moe_gated_ffn": ([_I] * 4 + [_P] * 10 + [_P, _SZ, _P], ctypes.c_int),
    "moe_gated_ffn_backward": ([_I] * 3 + [_P] * 9 + [_I] + [_P] * 2 + [_I] + [_P] * 4 + [_P, _SZ, _P],
                               ctypes.c_int),
    "moe_newton_schulz_workspace_bytes": ([_I] * 3, _SZ),
    "moe_newton_schulz": ([_I] * 4 + [_P, _I, _P, _I, _P, _F, _P, _SZ, _P], ctypes.c_int),
    "moe_muon_step": ([_I] * 3 + [_P] * 5 + [_F] * 3 + [_I, _I, _P, _F, _P, _SZ, _P], ctypes.c_int),
}
for _name, (_args, _res) in _SIG.items():
    _f = getattr(_lib, _name)
    _f.argtypes = _args
    _f.restype = _res

_ACT = {"silu": 0, "gelu": 1, "relu": 2}  # moe_act


# ------------------------------------------------------------ gated FFN --

def gated_ffn_workspace_bytes(T, d, h):
    return int(_lib.moe_gated_ffn_workspace_bytes(T, d, h))


def gated_ffn_backward_workspace_bytes(T, d, h):
    return int(_lib.moe_gated_ffn_backward_workspace_bytes(T, d, h))


def _ffn_sizes(x, w_gate, w_up, w_down):
    """T, d, h of x [T, d], w_gate and w_up [h, d], w_down [d, h]."""
    try:
        (T, d), (h, dg) = x.shape, w_gate.shape
        if dg == d and w_up.shape == w_gate.shape and w_down.shape == (d, h):
            return T, d, h
    except (AttributeError, ValueError):
        pass
    if not isinstance(x, torch.Tensor) or x.dim() != 2:
        raise ValueError("x: expected [T, d]")
    d = x.shape[1]
    if not isinstance(w_gate, torch.Tensor) or w_gate.dim() != 2:
        raise ValueError(f"w_gate: expected [h, {d}]")
    h, dg = w_gate.shape
    if dg != d:
        raise ValueError(f"w_gate: expected [h, {d}], got [{h}, {dg}]")
    _shape(w_up, "w_up", (h, d))
    _shape(w_down, "w_down", (d, h))


def _ptr(t, dtype, name, dev):
    """_arg of a tensor whose shape has been compared: its elements are not counted again
    (one token's call is bound by the host, which each question costs 0.1 to 0.2 us)."""
    if t is not None and t.dtype is dtype and t.get_device() == dev and t.is_contiguous():
        return t.data_ptr()
    return _arg(t, dtype, name, 0, dev)


def _shape(t, name, want):
    """Refuses a t that has not the shape want."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name}: expected a torch.Tensor")
    if t.shape != want:
        raise ValueError(f"{name}: expected {list(want)}, got {list(t.shape)}")


def gated_ffn(x, w_gate, w_up, w_down, add, token_scale, y, h_act, p_save, q_save, ws, act="silu",
              stream=None):
    """y = add + token_scale * (act(x Wg^T) * (x Wu^T)) Wd^T (include/moe_dense.h).  x [T, d],
    w_gate, w_up [h, d], w_down [d, h]; add, token_scale, and p_save with q_save may be None;
    act is "silu", "gelu" (the tanh form) or "relu"."""
    T, d, h = _ffn_sizes(x, w_gate, w_up, w_down)
    if act not in _ACT:
        raise ValueError(f"act: expected one of {', '.join(_ACT)}, got {act!r}")
    dev, n, nh = torch.cuda.current_device(), T * d, T * h
    wp, wn = _ws(ws, dev)
    _check(_lib.moe_gated_ffn(
        T, d, h, _ACT[act], _arg(x, _bf16, "x", n, dev), _ptr(w_gate, _bf16, "w_gate", dev),
        _ptr(w_up, _bf16, "w_up", dev), _ptr(w_down, _bf16, "w_down", dev),
        _arg(add, _bf16, "add", n, dev), _arg(token_scale, _f32, "token_scale", T, dev),
        _arg(y, _bf16, "y", n, dev), _arg(h_act, _bf16, "h_act", nh, dev),
        _arg(p_save, _bf16, "p_save", nh, dev), _arg(q_save, _bf16, "q_save", nh, dev), wp, wn,
        _on(stream, dev)), "moe_gated_ffn")


def gated_ffn_backward(x, w_gate, w_up, w_down, token_scale, h_act, p_save, q_save, dy, dx_in, dx,
                       dw_gate, dw_up, dw_down, dtoken_scale, ws, stream=None):
    """The backward of gated_ffn (include/moe_dense.h): dx = dx_in + the block's input gradient
    (bf16 or fp32, dx_in of dx's type or None), the weights' gradients and dtoken_scale (or
    None), all four bf16 or fp32."""
    T, d, h = _ffn_sizes(x, w_gate, w_up, w_down)
    xt, wt = _float_type(dx, "dx"), _float_type(dw_gate, "dw_gate")
    _shape(dw_gate, "dw_gate", (h, d))
    _shape(dw_up, "dw_up", (h, d))
    _shape(dw_down, "dw_down", (d, h))
    dev, n, nh = torch.cuda.current_device(), T * d, T * h
    wp, wn = _ws(ws, dev)
    _check(_lib.moe_gated_ffn_backward(
        T, d, h, _arg(x, _bf16, "x", n, dev), _ptr(w_gate, _bf16, "w_gate", dev),
        _ptr(w_up, _bf16, "w_up", dev), _ptr(w_down, _bf16, "w_down", dev),
        _arg(token_scale, _f32, "token_scale", T, dev), _arg(h_act, _bf16, "h_act", nh, dev),
        _arg(p_save, _bf16, "p_save", nh, dev), _arg(q_save, _bf16, "q_save", nh, dev),
        _arg(dy, _bf16, "dy", n, dev), _DTYPE[xt], _arg(dx_in, xt, "dx_in", n, dev),
        _arg(dx, xt, "dx", n, dev), _DTYPE[wt], _ptr(dw_gate, wt, "dw_gate", dev),
        _ptr(dw_up, wt, "dw_up", dev), _ptr(dw_down, wt, "dw_down", dev),
        _arg(dtoken_scale, wt, "dtoken_scale", T, dev), wp, wn, _on(stream, dev)),
        "moe_gated_ffn_backward")


# ------------------------------------------------------------ Newton-Schulz --

def newton_schulz_workspace_bytes(B, rows, cols):
    return int(_lib.moe_newton_schulz_workspace_bytes(B, rows, cols))


def _matrices(t, name):
    if not isinstance(t, torch.Tensor) or t.dim() not in (2, 3):
        raise ValueError(f"{name}: expected [B, rows, cols] or [rows, cols]")
    return (1, *t.shape) if t.dim() == 2 else tuple(t.shape)


def _same_matrices(t, name, want):
    """Refuses a t of other matrices than want's (None: left out)."""
    if t is None:
        return
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name}: expected a torch.Tensor")
    if t.shape != want.shape and _matrices(t, name) != _matrices(want, name):
        raise ValueError(f"{name}: expected {list(want.shape)}, got {list(t.shape)}")


def _coefficients(c, steps):
    """A float array of one (a, b, c) a step, or None: c is one triple for all steps, or one
    for each."""
    if c is None:
        return None
    rows = [list(t) if getattr(t, "ndim", 1) and hasattr(t, "__iter__") else [t] for t in c]
    c = [float(v) for t in rows for v in t]
    if len(c) == 3:
        c = c * steps
    if len(c) != 3 * steps:
        raise ValueError(f"coefficients: {len(c)} numbers, 3 or {3 * steps} expected")
    return (ctypes.c_float * len(c))(*c)


def newton_schulz(x, out, ws, steps=5, coefficients=None, eps=1e-7, stream=None):
    """out = x's matrices with their singular values taken to about 1 (include/moe_dense.h).
    x [B, rows, cols] or [rows, cols], bf16 or fp32, out of its shape (and x itself where the
    types are one); coefficients: one (a, b, c) for all steps, one for each, or None."""
    B, rows, cols = _matrices(x, "x")
    xt, ot = _float_type(x, "x"), _float_type(out, "out")
    _same_matrices(out, "out", x)
    dev = torch.cuda.current_device()
    wp, wn = _ws(ws, dev)
    _check(_lib.moe_newton_schulz(B, rows, cols, _DTYPE[xt], _ptr(x, xt, "x", dev), _DTYPE[ot],
                                  _ptr(out, ot, "out", dev), steps, _coefficients(coefficients, steps),
                                  eps, wp, wn, _on(stream, dev)), "moe_newton_schulz")


def muon_step(w, w_copy, momentum, grad, lr, mu, weight_decay, scale, ws, nesterov=True, steps=5,
              coefficients=None, eps=1e-7, stream=None):
    """One Muon step of w [B, rows, cols] or [rows, cols] (include/moe_dense.h): momentum and w
    fp32 in place, w_copy (or None) its bf16 copy, lr a [1] fp32 tensor on the device."""
    B, rows, cols = _matrices(w, "w")
    for t, name in ((w_copy, "w_copy"), (momentum, "momentum"), (grad, "grad")):
        _same_matrices(t, name, w)
    dev = torch.cuda.current_device()
    wp, wn = _ws(ws, dev)
    _check(_lib.moe_muon_step(
        B, rows, cols, _ptr(w, _f32, "w", dev), _ptr(w_copy, _bf16, "w_copy", dev),
        _ptr(momentum, _f32, "momentum", dev), _ptr(grad, _f32, "grad", dev),
        _arg(lr, _f32, "lr", 1, dev), mu, weight_decay, scale, 1 if nesterov else 0, steps,
        _coefficients(coefficients, steps), eps, wp, wn, _on(stream, dev)), "moe_muon_step")


# ------------------------------------------------------------- shared expert --

class SharedExpert:
    """A shared expert of a block (block_forward's and block_backward's `shared`): its bf16
    weights w_gate, w_up [h, d] and w_down [d, h], what its forward keeps for the backward
    (three [T, h] bf16 buffers and the token scale), and the gradients, which hold the last
    backward's results: dw_gate, dw_up, dw_down and, with a token scale, dtoken_scale,
    all fp32.  The next forward overwrites what it keeps: an expert that several blocks
    share runs each block's backward before the next block's forward."""

    def __init__(self, T, w_gate, w_up, w_down, act="silu"):
        h, d = w_gate.shape
        e = dict(device=w_gate.device)
        self.T, self.act = T, act
        self.w_gate, self.w_up, self.w_down = w_gate, w_up, w_down
        self.h_act, self.p_save, self.q_save = (torch.empty((T, h), dtype=_bf16, **e) for _ in range(3))
        self.saved = False                             # whether a forward has run
        self.forwards = 0                              # forwards begun, for the blocks that use it
        self.token_scale = None                        # scale, or None where every token's is 1
        self.scale = torch.empty(T, **e)
        self.dw_gate, self.dw_up = (torch.empty((h, d), **e) for _ in range(2))
        self.dw_down = torch.empty((d, h), **e)
        self.dtoken_scale = torch.empty(T, **e)
        n = max(gated_ffn_workspace_bytes(T, d, h), gated_ffn_backward_workspace_bytes(T, d, h), 256)
        self.ws = torch.zeros(n, dtype=torch.uint8, **e)

    def forward(self, x, add, y, token_scale=None, stream=None):
        """y = add + token_scale * expert(x); y may be add.  token_scale [T] fp32 (or None: 1)
        is copied for the backward."""
        if not isinstance(x, torch.Tensor) or x.dim() != 2 or x.shape[0] != self.T:
            raise ValueError(f"x: expected [{self.T}, d]")
        self.refuse_scale(token_scale)
        # from here on what the forward before kept is gone
        self.saved = False
        self.forwards += 1
        self.token_scale = None
        if token_scale is not None:
            self.token_scale = _keep(self.scale, token_scale.view(-1)[:self.T], stream)
        gated_ffn(x, self.w_gate, self.w_up, self.w_down, add, self.token_scale, y, self.h_act,
                  self.p_save, self.q_save, self.ws, self.act, stream)
        self.saved = True

    def refuse_scale(self, token_scale):
        """Raises if token_scale is not None nor T fp32 values on the current device."""
        if token_scale is not None:
            _arg(token_scale, _f32, "token_scale", self.T, torch.cuda.current_device())

    def backward(self, x, dy, dx_in, dx, stream=None):
        """dx = dx_in + the gradient of the forward's x (which x is), and the weights'."""
        if not self.saved:
            raise RuntimeError("backward of a shared expert without a forward")
        if not isinstance(x, torch.Tensor) or x.dim() != 2 or x.shape[0] != self.T:
            raise ValueError(f"x: expected [{self.T}, d]")
        gated_ffn_backward(x, self.w_gate, self.w_up, self.w_down, self.token_scale, self.h_act,
                           self.p_save, self.q_save, dy, dx_in, dx, self.dw_gate, self.dw_up,
                           self.dw_down, None if self.token_scale is None else self.dtoken_scale,
                           self.ws, stream)


# ------------------------------------------------------------------- Muon --

class Muon:
    """Muon over weight matrices.  weights: (w, w_copy) pairs, w [B, rows, cols] or
    [rows, cols] fp32 and w_copy its bf16 copy that the layer reads, or None.  lr is a [1]
    fp32 tensor on the device, which a schedule may fill between steps; scale multiplies the
    orthogonal factor (None: sqrt(max(1, rows / cols)) of each).  All steps run on one stream:
    the workspace is one for all weights."""

    def __init__(self, weights, lr=0.02, mu=0.95, weight_decay=0.0, nesterov=True, steps=5,
                 coefficients=None, scale=None, eps=1e-7):
        self.weights = list(weights)
        if not self.weights:
            raise ValueError("weights: none given")
        dev = self.weights[0][0].device
        self.momentum = [torch.zeros_like(w) for w, _ in self.weights]
        self.lr = torch.tensor([lr], dtype=_f32, device=dev)
        self.mu, self.weight_decay, self.nesterov, self.steps = mu, weight_decay, nesterov, steps
        self.coefficients, self.scale, self.eps = coefficients, scale, eps
        n = max(newton_schulz_workspace_bytes(*_matrices(w, "w")) for w, _ in self.weights)
        self.ws = torch.zeros(max(n, 256), dtype=torch.uint8, device=dev)

    def step(self, grads, stream=None):
        """One step of every weight; grads: fp32 tensors of the weights' shapes, in order."""
        grads = list(grads)
        if len(grads) != len(self.weights):
            raise ValueError(f"grads: {len(grads)} tensors, {len(self.weights)} weights")
        for i, ((w, _), g) in enumerate(zip(self.weights, grads)):  # before any weight moves
            _same_matrices(g, f"grads[{i}]", w)
        for (w, copy), v, g in zip(self.weights, self.momentum, grads):
            rows, cols = w.shape[-2:]
            scale = max(1.0, rows / cols) ** 0.5 if self.scale is None else self.scale
            muon_step(w, copy, v, g, self.lr, self.mu, self.weight_decay, scale, self.ws, self.nesterov,
                      self.steps, self.coefficients, self.eps, stream)
