"""Gated experts: both projections, the activation and their product in one kernel.

    p = cbd.expert_plan(t, e, c, 2 * k)                       # gate and other projection, W [E, 2K, C]
    d = cbd.expert_plan(t, e, k, c)                           # the last projection, D [E, C, K]
    h, gu = cbd.expert_gated_forward(p, x, w, ends, save=True)
    y = cbd.expert_forward(d, h, down, ends)
    dgu = cbd.expert_gated_bwd(d, dy, down, gu, ends)         # what reaches g and u
    dx, dw = cbd.expert_bwd_data(p, dgu, w, ends), cbd.expert_bwd_weight(p, dgu, x, ends)
    ddown = cbd.expert_bwd_weight(d, dy, h, ends)

h[t] = act(g) * u with (g, u) = gu[t] = W_e x[t], g in the first half of W's
outputs.  `expert_ffn(x, w, down, ends)` is all of it, differentiable.  Rows,
`ends`, layouts, strides and streams are those of the expert products;
include/cbd.h states the operation in full.

The two calls themselves are not recorded by autograd: where an operand
requires gradients they are refused, and `expert_ffn` is the way.
"""
from __future__ import annotations

import ctypes
import functools

from . import _check, _lib
from .experts import (_DENSE, ExpertInfo, ExpertPlan, _any_records, _cached, _ends, _handle, _on, _strided, _w_layout,
                      _written, expert_bwd_data, expert_bwd_weight, expert_forward)

ACT_SILU, ACT_GELU, ACT_RELU = 0, 1, 2
_ACTS = {"silu": ACT_SILU, "gelu": ACT_GELU, "relu": ACT_RELU}


class GatedStrides(ctypes.Structure):
    _fields_ = [("in_row", ctypes.c_int64), ("h_row", ctypes.c_int64), ("gu_row", ctypes.c_int64),
                ("dgu_row", ctypes.c_int64), ("w_row", ctypes.c_int64), ("w_expert", ctypes.c_int64)]


def _bind():
    P = ctypes.POINTER
    V = ctypes.c_void_p
    _lib.cbd_expert_gated_forward.argtypes = [V, V, V, V, V, V, ctypes.c_int32, P(GatedStrides), V]
    _lib.cbd_expert_gated_bwd.argtypes = [V, V, V, V, V, V, ctypes.c_int32, P(GatedStrides), V]
    _lib.cbd_expert_gated_info.argtypes = [V, ctypes.c_int32, P(ExpertInfo)]
    for f in ("forward", "bwd", "info"):
        getattr(_lib, "cbd_expert_gated_" + f).restype = ctypes.c_int


_bind()


def _act(v):
    if isinstance(v, str):
        if v not in _ACTS:
            raise ValueError(f"unknown activation {v!r}; one of {sorted(_ACTS)}")
        return _ACTS[v]
    return int(v)


def _hidden(p):
    if p.k % 2:
        raise ValueError(f"the plan's k is {p.k}: two projections need an even one")
    return p.k // 2


def _refuse(name, *operands):
    if _any_records(operands):
        raise ValueError(f"{name} is not recorded by autograd and an operand requires gradients (or has a "
                         "tangent); use expert_ffn or call under torch.no_grad()")


def _given(t, shape, dtype, device, name):
    """An output and its strides: allocated, or the caller's."""
    import torch

    if t is None:
        return torch.empty(shape, dtype=dtype, device=device), _DENSE[2]
    s = _strided(t, shape, dtype, device, name)
    _written(t)
    return t, s


def _gated_strides(s_in, s_h, s_gu, s_dgu, s_w):
    if s_in is s_h is s_gu is s_dgu is _DENSE[2] and s_w is _DENSE[3]:
        return None
    return ctypes.byref(GatedStrides(s_in[0], s_h[0], s_gu[0], s_dgu[0], s_w[1], s_w[0]))


def expert_gated_forward(p: ExpertPlan, x, w, ends, act="silu", save=False, h=None, gu=None, stream=None):
    """h[t] = act(g) * u on `stream` (default: torch's current one); with save,
    or a given gu, (h, gu) with gu[t] = (g, u).  p is the plan of both
    projections (k = 2 K); outputs are allocated unless given."""
    _refuse("expert_gated_forward", x, w)
    k, act = _hidden(p), _act(act)
    s_x = _strided(x, (p.tokens, p.c), p._tdtype, None, "x")
    dev = x.device
    s_w = _strided(w, p.w_shape, p._tdtype, dev, "w")
    bits = _ends(p, ends, dev)
    with _on(dev, stream):
        h, s_h = _given(h, (p.tokens, k), p._tdtype, dev, "h")
        s_gu = _DENSE[2]
        if save or gu is not None:
            gu, s_gu = _given(gu, (p.tokens, 2 * k), p._tdtype, dev, "gu")
        _check(_lib.cbd_expert_gated_forward(p._h[bits], x.data_ptr(), w.data_ptr(), ends.data_ptr(), h.data_ptr(),
                                             None if gu is None else gu.data_ptr(), act,
                                             _gated_strides(s_x, s_h, s_gu, _DENSE[2], s_w), _handle(stream, dev)),
               "cbd_expert_gated_forward")
    return h if gu is None else (h, gu)


def expert_gated_bwd(p: ExpertPlan, dy, w, gu, ends, act="silu", dgu=None, stream=None):
    """dgu[t] = (dh * u * act'(g), dh * act(g)) with dh = D_e^T dy[t] and (g, u)
    = gu[t]; p is the plan of the last projection D, w its weights."""
    _refuse("expert_gated_bwd", dy, w, gu)
    act = _act(act)
    s_dy = _strided(dy, (p.tokens, p.k), p._tdtype, None, "dy")
    dev = dy.device
    s_w = _strided(w, p.w_shape, p._tdtype, dev, "w")
    s_gu = _strided(gu, (p.tokens, 2 * p.c), p._tdtype, dev, "gu")
    bits = _ends(p, ends, dev)
    with _on(dev, stream):
        dgu, s_dgu = _given(dgu, (p.tokens, 2 * p.c), p._tdtype, dev, "dgu")
        _check(_lib.cbd_expert_gated_bwd(p._h[bits], dy.data_ptr(), w.data_ptr(), gu.data_ptr(), ends.data_ptr(),
                                         dgu.data_ptr(), act, _gated_strides(s_dy, _DENSE[2], s_gu, s_dgu, s_w),
                                         _handle(stream, dev)), "cbd_expert_gated_bwd")
    return dgu


def expert_gated_info(p: ExpertPlan, bwd=False) -> ExpertInfo:
    """What the call launches on dense, 16-byte aligned tensors."""
    out = ExpertInfo()
    _check(_lib.cbd_expert_gated_info(p._h[32], int(bool(bwd)), ctypes.byref(out)), "cbd_expert_gated_info")
    return out


@functools.lru_cache(None)
def _recorder():
    import torch

    class GatedExperts(torch.autograd.Function):
        @staticmethod
        def forward(ctx, x, w, down, ends, p, d, act):
            keep = any(ctx.needs_input_grad[:3])
            h, gu = (expert_gated_forward(p, x, w, ends, act, save=True) if keep
                     else (expert_gated_forward(p, x, w, ends, act), None))
            ctx.plans, ctx.act = (p, d), act
            if keep:
                # h is kept as the last projection read it, so that its weights'
                # gradient is that of what was computed.
                ctx.save_for_backward(x, w, down, ends, gu, h if ctx.needs_input_grad[2] else None)
            return expert_forward(d, h, down, ends)

        @staticmethod
        @torch.autograd.function.once_differentiable
        def backward(ctx, dy):
            (p, d), (x, w, down, ends, gu, h) = ctx.plans, ctx.saved_tensors
            need_x, need_w, need_down = ctx.needs_input_grad[:3]
            dy = dy.contiguous()
            dx = dw = ddown = None
            if need_x or need_w:
                dgu = expert_gated_bwd(d, dy, down, gu, ends, ctx.act)
                dx = expert_bwd_data(p, dgu, w, ends) if need_x else None
                dw = expert_bwd_weight(p, dgu, x, ends) if need_w else None
            if need_down:
                ddown = expert_bwd_weight(d, dy, h, ends)
            return dx, dw, ddown, None, None, None, None

    return GatedExperts


def expert_ffn(x, w, down, ends, act="silu", w_layout="ekc"):
    """y[t] = D_e (act(G_e x[t]) * (U_e x[t])): x [T, C], w [E, 2K, C] or [E, C,
    2K] with the gate's half first, down [E, C, K] or [E, K, C] in the same
    layout.  Differentiable once in x, w and down.  The gradients between the
    products are in the operands' type, as h and y are."""
    if x.dim() != 2 or w.dim() != 3 or down.dim() != 3:
        raise ValueError("x must be [T, C], w and down have three dimensions")
    p = _cached(x.shape[0], tuple(w.shape), w_layout, w.dtype, None)
    d = _cached(x.shape[0], tuple(down.shape), _w_layout(w_layout), down.dtype, None)
    if (d.experts, d.c, d.k) != (p.experts, _hidden(p), p.c) or w.dtype != down.dtype:
        raise ValueError(f"w {tuple(w.shape)} {w.dtype} and down {tuple(down.shape)} {down.dtype} do not fit together")
    if not x.is_cuda:
        raise ValueError("x must be a GPU torch tensor")
    # The node belongs to the tensors' device and the current stream there.
    with _on(x.device, None):
        return _recorder().apply(x, w, down, ends, p, d, _act(act))
