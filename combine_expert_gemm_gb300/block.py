"""Python binding of the operators around the routed-expert layer in a
pre-norm training block (``include/moe_block.h``): layer norm, the router's
balance loss with the dense router gradient, and 8-bit activation checkpoints.

Argument marshalling only, as in the package's ``__init__``; these calls also
compare every tensor's size with the shape, because a short buffer would be
overrun on the device.
"""
import contextlib
import ctypes

import torch

from . import (_P, _SP, _SZ, BackwardBuffers, LayerBuffers, _bf16, _check, _current_raw_stream, _f32, _i32,
               _lib, _stream, _u8, combine, dispatch, dispatch_backward, expert_ffn, expert_ffn_backward, route,
               route_logits, route_workspace_bytes)

__all__ = ["layer_norm", "layer_norm_backward", "layer_norm_backward_workspace_bytes",
           "balance_loss", "balance_loss_backward", "balance_loss_workspace_bytes",
           "router_dense_backward", "router_dense_backward_workspace_bytes",
           "checkpoint_save", "checkpoint_restore", "combine_backward_checkpoint", "BlockState",
           "BlockScratch", "block_forward", "block_backward"]

_I = ctypes.c_int32
_SIG = {
    "moe_layer_norm": ([_I] * 3 + [_P] * 4 + [ctypes.c_float] + [_P] * 4 + [_P], ctypes.c_int),
    "moe_layer_norm_backward_workspace_bytes": ([_I, _I], _SZ),
    "moe_layer_norm_backward": ([_I] * 3 + [_P, _I] + [_P] * 4 + [_I] + [_P] * 4 + [_P, _SZ, _P],
                                ctypes.c_int),
    "moe_balance_loss_workspace_bytes": ([_SP], _SZ),
    "moe_balance_loss": ([_SP] + [_P] * 8 + [_P, _SZ, _P], ctypes.c_int),
    "moe_balance_loss_backward": ([_SP] + [_P] * 9 + [_P], ctypes.c_int),
    "moe_router_dense_backward_workspace_bytes": ([_SP], _SZ),
    "moe_router_dense_backward": ([_SP] + [_P] * 7 + [_P, _SZ, _P], ctypes.c_int),
    "moe_checkpoint_save": ([_SP] + [_P] * 10 + [_P], ctypes.c_int),
    "moe_checkpoint_restore": ([_SP] + [_P] * 8 + [_P], ctypes.c_int),
    "moe_combine_backward_checkpoint": ([_SP] + [_P] * 8 + [_P], ctypes.c_int),
}
for _name, (_args, _res) in _SIG.items():
    _f = getattr(_lib, _name)
    _f.argtypes = _args
    _f.restype = _res

_DTYPE = {torch.bfloat16: 0, torch.float32: 1}  # moe_dtype
_i8 = torch.int8


def _arg(t, dtype, name, n, dev):
    """Device pointer of a contiguous CUDA tensor of n elements (None: NULL)."""
    if t is None:
        return None
    # the calls are short: a good tensor is passed with as few steps as the
    # checks need, and only a bad one is asked what is wrong with it
    try:
        if t.dtype is dtype and t.get_device() == dev and t.is_contiguous() and t.numel() >= n:
            return t.data_ptr()
    except AttributeError:
        pass
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name}: expected a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name}: must be a CUDA tensor")
    if t.get_device() != dev:
        raise ValueError(f"{name}: on {t.device}, but the current device is cuda:{dev}")
    if t.dtype is not dtype:
        raise TypeError(f"{name}: expected {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name}: must be contiguous")
    raise ValueError(f"{name}: {t.numel()} elements, {n} needed")


def _on(stream, dev):
    """The stream's handle; the current stream of the current device dev by default."""
    if stream is None and _current_raw_stream is not None:
        return _current_raw_stream(dev)
    return _stream(stream)


def _ws(ws, dev):
    p = _arg(ws, _u8, "ws", 0, dev)
    return p, 0 if ws is None else ws.numel()


def _float_type(t, name):
    if not isinstance(t, torch.Tensor) or t.dtype not in _DTYPE:
        raise TypeError(f"{name}: expected a bfloat16 or float32 tensor")
    return t.dtype


def _rows(x, name):
    dt = _float_type(x, name)
    if x.dim() != 2:
        raise ValueError(f"{name}: expected [rows, d]")
    rows, d = x.shape
    return dt, rows, d


# -------------------------------------------------------------- layer norm --

def layer_norm(x, add, gamma, beta, eps, x_sum, y, mean, rstd, stream=None):
    """x_sum = x + add and y = layer norm of it (include/moe_block.h).  x [rows, d]
    bf16 or fp32; add and x_sum, gamma, beta, and mean with rstd may be None."""
    dt, rows, d = _rows(x, "x")
    dev, n = torch.cuda.current_device(), rows * d
    _check(_lib.moe_layer_norm(
        rows, d, _DTYPE[dt], _arg(x, dt, "x", n, dev), _arg(add, _bf16, "add", n, dev),
        _arg(gamma, _f32, "gamma", d, dev), _arg(beta, _f32, "beta", d, dev), eps,
        _arg(x_sum, dt, "x_sum", n, dev), _arg(y, _bf16, "y", n, dev),
        _arg(mean, _f32, "mean", rows, dev), _arg(rstd, _f32, "rstd", rows, dev), _on(stream, dev)),
        "moe_layer_norm")


def layer_norm_backward_workspace_bytes(rows, d):
    return int(_lib.moe_layer_norm_backward_workspace_bytes(rows, d))


def layer_norm_backward(x, dy, gamma, mean, rstd, dres, dx, dgamma, dbeta, ws, stream=None):
    """dx = dres + the norm's input gradient, dgamma, dbeta (include/moe_block.h).  x and
    dy are bf16 or fp32 each, dres and dx of one type; gamma, dres, dgamma and dbeta may
    be None."""
    dt, rows, d = _rows(x, "x")
    yt, gt = _float_type(dy, "dy"), _float_type(dx, "dx")
    dev, n = torch.cuda.current_device(), rows * d
    wp, wn = _ws(ws, dev)
    _check(_lib.moe_layer_norm_backward(
        rows, d, _DTYPE[dt], _arg(x, dt, "x", n, dev), _DTYPE[yt], _arg(dy, yt, "dy", n, dev),
        _arg(gamma, _f32, "gamma", d, dev), _arg(mean, _f32, "mean", rows, dev),
        _arg(rstd, _f32, "rstd", rows, dev), _DTYPE[gt], _arg(dres, gt, "dres", n, dev),
        _arg(dx, gt, "dx", n, dev), _arg(dgamma, _f32, "dgamma", d, dev),
        _arg(dbeta, _f32, "dbeta", d, dev), wp, wn, _on(stream, dev)), "moe_layer_norm_backward")


# ------------------------------------------------------------ balance loss --

def balance_loss_workspace_bytes(shape):
    return int(_lib.moe_balance_loss_workspace_bytes(ctypes.byref(shape)))


def balance_loss(shape, logits, topk_idx, token_mask, expert_count, token_count, expert_prob, lse,
                 losses, ws, stream=None):
    """losses = (balance loss, z loss) with the counts, mean probabilities and log sums
    that their gradient needs (include/moe_block.h).  token_mask [T] uint8 or None."""
    T, N, K = shape.T, shape.N, shape.K
    dev = torch.cuda.current_device()
    wp, wn = _ws(ws, dev)
    _check(_lib.moe_balance_loss(
        ctypes.byref(shape), _arg(logits, _f32, "logits", T * N, dev),
        _arg(topk_idx, _i32, "topk_idx", T * K, dev), _arg(token_mask, _u8, "token_mask", T, dev),
        _arg(expert_count, _i32, "expert_count", N, dev),
        _arg(token_count, _i32, "token_count", 1, dev),
        _arg(expert_prob, _f32, "expert_prob", N, dev), _arg(lse, _f32, "lse", T, dev),
        _arg(losses, _f32, "losses", 2, dev), wp, wn, _on(stream, dev)), "moe_balance_loss")


def balance_loss_backward(shape, logits, topk_idx, token_mask, expert_count, token_count, lse,
                          dlosses, dlogit, dlogits, stream=None):
    """dlogits [T, N] of both losses, plus the gates' dlogit [T, K] (or None) at the chosen
    experts (include/moe_block.h)."""
    T, N, K = shape.T, shape.N, shape.K
    dev = torch.cuda.current_device()
    _check(_lib.moe_balance_loss_backward(
        ctypes.byref(shape), _arg(logits, _f32, "logits", T * N, dev),
        _arg(topk_idx, _i32, "topk_idx", T * K, dev), _arg(token_mask, _u8, "token_mask", T, dev),
        _arg(expert_count, _i32, "expert_count", N, dev),
        _arg(token_count, _i32, "token_count", 1, dev), _arg(lse, _f32, "lse", T, dev),
        _arg(dlosses, _f32, "dlosses", 2, dev), _arg(dlogit, _f32, "dlogit", T * K, dev),
        _arg(dlogits, _f32, "dlogits", T * N, dev), _on(stream, dev)), "moe_balance_loss_backward")


def router_dense_backward_workspace_bytes(shape):
    return int(_lib.moe_router_dense_backward_workspace_bytes(ctypes.byref(shape)))


def router_dense_backward(shape, x, w_router, dlogits, dx_in, dx, dw_router, dbias, ws,
                          stream=None):
    """dx = dx_in + dlogits W, dw_router = dlogits^T x, dbias = column sums; dx_in may be
    None or dx itself, and each output may be None (include/moe_block.h)."""
    T, d, N = shape.T, shape.d, shape.N
    dev = torch.cuda.current_device()
    wp, wn = _ws(ws, dev)
    _check(_lib.moe_router_dense_backward(
        ctypes.byref(shape), _arg(x, _bf16, "x", T * d, dev),
        _arg(w_router, _f32, "w_router", N * d, dev), _arg(dlogits, _f32, "dlogits", T * N, dev),
        _arg(dx_in, _f32, "dx_in", T * d, dev), _arg(dx, _f32, "dx", T * d, dev),
        _arg(dw_router, _f32, "dw_router", N * d, dev), _arg(dbias, _f32, "dbias", N, dev), wp, wn,
        _on(stream, dev)), "moe_router_dense_backward")


# ------------------------------------------------------- 8-bit checkpoints --

def checkpoint_save(shape, expert_offset, g_save, u_save, y_disp, g_q, g_scale, u_q, u_scale, y_q,
                    y_scale, stream=None):
    """The valid rows of g_save, u_save and y_disp in MXINT8 (include/moe_block.h); a
    source that is None is left out."""
    h, d, R = shape.h, shape.d, shape.R
    dev = torch.cuda.current_device()
    _check(_lib.moe_checkpoint_save(
        ctypes.byref(shape), _arg(expert_offset, _i32, "expert_offset", shape.N + 1, dev),
        _arg(g_save, _bf16, "g_save", R * h, dev), _arg(u_save, _bf16, "u_save", R * h, dev),
        _arg(y_disp, _bf16, "y_disp", R * d, dev), _arg(g_q, _i8, "g_q", R * h, dev),
        _arg(g_scale, _u8, "g_scale", R * h // 32, dev), _arg(u_q, _i8, "u_q", R * h, dev),
        _arg(u_scale, _u8, "u_scale", R * h // 32, dev), _arg(y_q, _i8, "y_q", R * d, dev),
        _arg(y_scale, _u8, "y_scale", R * d // 32, dev), _on(stream, dev)), "moe_checkpoint_save")


def checkpoint_restore(shape, expert_offset, g_q, g_scale, u_q, u_scale, g_save, u_save, h_act,
                       stream=None):
    """g_save, u_save and h_act = silu(G) U of a checkpoint (include/moe_block.h)."""
    n, dev = shape.R * shape.h, torch.cuda.current_device()
    _check(_lib.moe_checkpoint_restore(
        ctypes.byref(shape), _arg(expert_offset, _i32, "expert_offset", shape.N + 1, dev),
        _arg(g_q, _i8, "g_q", n, dev), _arg(g_scale, _u8, "g_scale", n // 32, dev),
        _arg(u_q, _i8, "u_q", n, dev), _arg(u_scale, _u8, "u_scale", n // 32, dev),
        _arg(g_save, _bf16, "g_save", n, dev), _arg(u_save, _bf16, "u_save", n, dev),
        _arg(h_act, _bf16, "h_act", n, dev), _on(stream, dev)), "moe_checkpoint_restore")


def combine_backward_checkpoint(shape, dy, y_q, y_scale, route_row, topk_gate, dy_disp, dgate,
                                dlogit=None, stream=None):
    """combine_backward with y_disp read from its checkpoint, and the chosen logits'
    gradient into dlogit [T, K] if given (include/moe_block.h)."""
    T, d, K, R = shape.T, shape.d, shape.K, shape.R
    dev = torch.cuda.current_device()
    _check(_lib.moe_combine_backward_checkpoint(
        ctypes.byref(shape), _arg(dy, _bf16, "dy", T * d, dev), _arg(y_q, _i8, "y_q", R * d, dev),
        _arg(y_scale, _u8, "y_scale", R * d // 32, dev),
        _arg(route_row, _i32, "route_row", T * K, dev),
        _arg(topk_gate, _f32, "topk_gate", T * K, dev), _arg(dy_disp, _bf16, "dy_disp", R * d, dev),
        _arg(dgate, _f32, "dgate", T * K, dev), _arg(dlogit, _f32, "dlogit", T * K, dev),
        _on(stream, dev)), "moe_combine_backward_checkpoint")


# ------------------------------------------------------------------- block --

class BlockState:
    """What one pre-norm block keeps from its forward to its backward: the residual
    stream, the norm's output and statistics, the routes, the router's logits and
    log sums, and the experts' buffers in 8 bits (33/32 bytes an element of G, U and
    y_disp).  The bf16 buffers of the experts live in a BlockScratch that every block
    of a model shares."""

    def __init__(self, shape, device="cuda"):
        T, d, N, K, h, R = shape.T, shape.d, shape.N, shape.K, shape.h, shape.R
        e = dict(device=device)
        self.shape = shape
        self.h = None                                  # the rows that were normalised: x_sum or x_fp32
        self.x_sum = torch.empty((T, d), dtype=_bf16, **e)
        self.x_fp32 = None                             # allocated by the first fp32 x
        self.n = torch.empty((T, d), dtype=_bf16, **e)
        self.mean, self.rstd = torch.empty(T, **e), torch.empty(T, **e)
        self.topk_idx = torch.empty((T, K), dtype=_i32, **e)
        self.topk_gate = torch.empty((T, K), **e)
        self.route_row = torch.empty((T, K), dtype=_i32, **e)
        self.expert_demand = torch.empty(N, dtype=_i32, **e)
        self.expert_count = torch.empty(N, dtype=_i32, **e)
        self.expert_offset = torch.empty(N + 1, dtype=_i32, **e)
        # the logits stay in moe_route's workspace
        self.route_ws = torch.zeros(max(route_workspace_bytes(shape), 256), dtype=_u8, **e)
        self.routed_count = torch.empty(N, dtype=_i32, **e)
        self.token_count = torch.empty(1, dtype=_i32, **e)
        self.expert_prob = torch.empty(N, **e)
        self.lse = torch.empty(T, **e)
        self.losses = torch.empty(2, **e)              # balance loss, z loss
        self.token_mask = None                         # mask, or None if every token counts
        self.mask = torch.empty(T, dtype=_u8, **e)
        self.g_q, self.u_q = (torch.empty((R, h), dtype=_i8, **e) for _ in range(2))
        self.g_scale, self.u_scale = (torch.empty((R, h // 32), dtype=_u8, **e) for _ in range(2))
        self.y_q = torch.empty((R, d), dtype=_i8, **e)
        self.y_scale = torch.empty((R, d // 32), dtype=_u8, **e)
        self.shared = None                             # the last forward's shared expert, and which
        self.shared_forward = 0                        # of that expert's forwards it was


class BlockScratch:
    """The buffers and workspaces that every block of one shape shares: the layer's
    forward and backward buffers (LayerBuffers, BackwardBuffers) and those of the norm,
    the balance loss and the dense router gradient.  `bwd` and the gradients below hold
    the last block_backward's results until the next one."""

    def __init__(self, shape, device="cuda"):
        T, d, N, K = shape.T, shape.d, shape.N, shape.K
        w = lambda n: torch.zeros(n, dtype=_u8, device=device)
        self.fwd = LayerBuffers(shape, device, save_for_backward=True)
        self.bwd = BackwardBuffers(shape, device)
        self.dgamma, self.dbeta = (torch.empty(d, device=device) for _ in range(2))
        self.dlogits = torch.empty((T, N), device=device)
        self.norm_ws = w(layer_norm_backward_workspace_bytes(T, d))
        self.balance_ws = w(balance_loss_workspace_bytes(shape))
        self.dense_ws = w(router_dense_backward_workspace_bytes(shape))


def _keep(dst, src, stream):
    """dst, or where it is None a new tensor of the calls' stream (on another one its
    memory could still be in use), with a copy of src made on that stream."""
    with contextlib.nullcontext() if stream is None else torch.cuda.stream(stream):
        if dst is None:
            dst = torch.empty_like(src)
        return dst.copy_(src)


def block_forward(st, sc, x, add, gamma, beta, w_router, bias, w_gate, w_up, w_down, eps=1e-5,
                  token_mask=None, stream=None, shared=None, shared_scale=None):
    """One pre-norm block: h = x + add (add: the previous block's output, or None),
    n = layer norm of h, and the routed-expert layer of n; its output is returned
    (sc.fwd.y, which the next block takes as add).  shared (a SharedExpert, or None) adds its
    own output of n, times shared_scale [T] fp32 where that is given.  st keeps what block_backward needs,
    the experts' buffers in 8 bits, and st.losses the balance and z loss over the tokens
    that token_mask [T] uint8 (or None: all) counts.  x, add and token_mask are copied
    where the backward needs them and may be overwritten once these calls have run.
    block_backward takes the same shared, before that runs another forward."""
    s, f = st.shape, sc.fwd
    _, rows, d = _rows(x, "x")
    if (rows, d) != (s.T, s.d):
        raise ValueError(f"x: expected [{s.T}, {s.d}], got [{rows}, {d}]")
    if shared is None:
        if shared_scale is not None:
            raise ValueError("shared_scale: given without shared")
    elif (shared.T, shared.w_gate.shape[1]) != (s.T, s.d):
        raise ValueError(f"shared: an expert of [{shared.T}, {shared.w_gate.shape[1]}], [{s.T}, {s.d}] expected")
    else:
        shared.refuse_scale(shared_scale)
    layer_norm(x, add, gamma, beta, eps, None if add is None else st.x_sum, st.n, st.mean, st.rstd,
               stream)
    st.shared = None
    if add is not None:
        st.h = st.x_sum
    elif x.dtype is _f32:
        st.h = st.x_fp32 = _keep(st.x_fp32, x, stream)
    else:
        st.h = _keep(st.x_sum, x, stream)
    route(s, st.n, w_router, bias, st.topk_idx, st.topk_gate, st.route_row, st.expert_count,
          st.expert_offset, st.expert_demand, st.route_ws, stream)
    balance_loss(s, route_logits(s, st.route_ws), st.topk_idx, token_mask, st.routed_count,
                 st.token_count, st.expert_prob, st.lse, st.losses, sc.balance_ws, stream)
    st.token_mask = None
    if token_mask is not None:
        st.token_mask = _keep(st.mask, token_mask.view(-1)[:s.T], stream)
    dispatch(s, st.n, st.route_row, f.x_disp, stream)
    expert_ffn(s, f.x_disp, st.expert_count, st.expert_offset, w_gate, w_up, w_down, f.h_act,
               f.g_save, f.u_save, f.y_disp, f.ffn_ws, stream)
    checkpoint_save(s, st.expert_offset, f.g_save, f.u_save, f.y_disp, st.g_q, st.g_scale, st.u_q,
                    st.u_scale, st.y_q, st.y_scale, stream)
    combine(s, f.y_disp, st.route_row, st.topk_gate, f.y, stream)
    if shared is not None:
        shared.forward(st.n, f.y, f.y, shared_scale, stream)
        st.shared, st.shared_forward = shared, shared.forwards
    return f.y


def block_backward(st, sc, dh, dx, dlosses, gamma, beta, w_router, bias, w_gate, w_up, w_down,
                   stream=None, shared=None):
    """The backward of block_forward.  dh [T, d] bf16 is the gradient of h + y (the next
    block's dx): it reaches h directly and through the layer.  dx [T, d] bf16 (dh itself
    is allowed) gets the gradient of h; dlosses [2] fp32 on the device are the gradients
    of st.losses.  sc.bwd.dw_gate, dw_up, dw_down, dw_router (and dbias), sc.dgamma and
    sc.dbeta hold the weights' gradients until the next call.  shared is the forward's; it
    holds its own weights' gradients."""
    if shared is not st.shared:
        raise ValueError("shared: this state's forward ran without one" if st.shared is None else
                         "shared: not the shared expert of this state's forward")
    if shared is not None and shared.forwards != st.shared_forward:
        raise RuntimeError("shared: another forward of this expert has run since this state's")
    s, f, b = st.shape, sc.fwd, sc.bwd
    combine_backward_checkpoint(s, dh, st.y_q, st.y_scale, st.route_row, st.topk_gate, b.dy_disp,
                                b.dgate, b.dlogit, stream)
    dispatch(s, st.n, st.route_row, f.x_disp, stream)
    checkpoint_restore(s, st.expert_offset, st.g_q, st.g_scale, st.u_q, st.u_scale, f.g_save,
                       f.u_save, f.h_act, stream)
    expert_ffn_backward(s, f.x_disp, st.expert_count, st.expert_offset, w_gate, w_up, w_down,
                        f.g_save, f.u_save, f.h_act, b.dy_disp, b.dx_disp, b.dw_gate, b.dw_up,
                        b.dw_down, b.ws, stream)
    dispatch_backward(s, b.dx_disp, st.route_row, b.dx, stream)
    if shared is not None:
        shared.backward(st.n, dh, b.dx, b.dx, stream)
    balance_loss_backward(s, route_logits(s, st.route_ws), st.topk_idx, st.token_mask,
                          st.routed_count, st.token_count, st.lse, dlosses, b.dlogit, sc.dlogits,
                          stream)
    router_dense_backward(s, st.n, w_router, sc.dlogits, b.dx, b.dx, b.dw_router,
                          None if bias is None else b.dbias, sc.dense_ws, stream)
    layer_norm_backward(st.h, b.dx, gamma, st.mean, st.rstd, dh, dx,
                        None if gamma is None else sc.dgamma, None if beta is None else sc.dbeta,
                        sc.norm_ws, stream)
    return dx
