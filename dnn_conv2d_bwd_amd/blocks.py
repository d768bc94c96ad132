"""The norms around a block, with its gate and residual.

    p = cbd.block_plan(rows, c, scale=0.5)
    z, n = cbd.block_forward(p, r, y, w_post=a, gate=g, w_pre=b)
    z, n, stats = cbd.block_forward(p, r, y, w_post=a, gate=g, w_pre=b, save=True)
    dr, dy, da, dg, db = cbd.block_bwd(p, dz, dn, r, y, stats, w_post=a, gate=g, w_pre=b)

z = r + scale * gate * (w_post * norm(y)) and n = w_pre * norm(z), with norm(v) =
v / sqrt(mean(v^2) + eps) over the last dimension: r is the residual stream, y
what a block made of it, n what the next block reads.  Every part but r may be
left out: without w_post y is not normed, without y there is only n, without
w_pre only z (None stands for what is not there).  The gate is one vector [C]
for all rows, or has a row for each, [T, C].

Where an operand requires gradients, block_forward is recorded by autograd (once
differentiable); `block_norm(r, y, ...)` makes the plan itself.  Tensors given
to be written to count as changed in place.  include/cbd.h states the operation
in full.
"""
from __future__ import annotations

import ctypes
import functools

from . import BF16, F32, _check, _dtype, _lib, _torch_dtype
from .experts import _DENSE, _any_records, _handle, _on, _strided, _written

GATE_NONE, GATE_CHANNEL, GATE_ROW = 0, 1, 2


class BlockProblem(ctypes.Structure):
    _fields_ = [("rows", ctypes.c_int64), ("c", ctypes.c_int64), ("dtype", ctypes.c_int32),
                ("dw_dtype", ctypes.c_int32), ("eps", ctypes.c_double), ("scale", ctypes.c_double)]


class BlockParams(ctypes.Structure):
    _fields_ = [("w_post", ctypes.c_void_p), ("gate", ctypes.c_void_p), ("w_pre", ctypes.c_void_p),
                ("gate_kind", ctypes.c_int32), ("reserved", ctypes.c_int32)]


class BlockStrides(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int64) for n in ("r", "y", "gate", "z", "n", "dz", "dn", "dr", "dy", "dgate")]


class BlockGrads(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in ("dr", "dy", "dw_post", "dgate", "dw_pre")]


def _bind():
    P = ctypes.POINTER
    V = ctypes.c_void_p
    U = ctypes.c_uint64
    _lib.cbd_block_plan.argtypes = [P(BlockProblem), P(V)]
    _lib.cbd_block_plan_destroy.argtypes = [V]
    _lib.cbd_block_plan_destroy.restype = None
    _lib.cbd_block_workspace_size.argtypes = [V, P(U)]
    _lib.cbd_block_forward.argtypes = [V, V, V, P(BlockParams), V, V, V, P(BlockStrides), V]
    _lib.cbd_block_bwd.argtypes = [V, V, V, V, V, V, P(BlockParams), P(BlockGrads), P(BlockStrides), V, U, V]
    for f in ("plan", "workspace_size", "forward", "bwd"):
        getattr(_lib, "cbd_block_" + f).restype = ctypes.c_int


_bind()


class BlockPlan:
    """Owns a cbd_block_plan_t; immutable; safe to run from several streams (a
    workspace each)."""

    def __init__(self, rows, c, dtype=BF16, dw_dtype=None, eps=1e-6, scale=1.0):
        self.rows, self.c, self.dtype = int(rows), int(c), _dtype(dtype)
        self.dw_dtype = self.dtype if dw_dtype is None else _dtype(dw_dtype)
        self.eps, self.scale = float(eps), float(scale)
        prob = BlockProblem(self.rows, self.c, self.dtype, self.dw_dtype, self.eps, self.scale)
        h = ctypes.c_void_p()
        _check(_lib.cbd_block_plan(ctypes.byref(prob), ctypes.byref(h)), "cbd_block_plan")
        self._h = h
        out = ctypes.c_uint64()
        _check(_lib.cbd_block_workspace_size(h, ctypes.byref(out)), "cbd_block_workspace_size")
        self._ws = int(out.value)
        self._tdtype, self._tdw = _torch_dtype(self.dtype), _torch_dtype(self.dw_dtype)
        self._shape, self._vshape = (self.rows, self.c), (self.c,)

    def workspace_size(self) -> int:
        """Bytes of device workspace the backward call needs."""
        return self._ws

    def __del__(self):
        h = getattr(self, "_h", None)
        lib = _lib  # None during interpreter shutdown
        if lib is not None and h is not None and h.value:
            lib.cbd_block_plan_destroy(h)
            self._h = None


def block_plan(rows, c, dtype="bf16", dw_dtype=None, eps=1e-6, scale=1.0) -> BlockPlan:
    """dw_dtype: type of the vectors' gradients (default: dtype)."""
    return BlockPlan(rows, c, dtype, dw_dtype, eps, scale)


def _vector(t, p, device, name):
    if (not hasattr(t, "data_ptr") or t.dtype is not p._tdtype or t.shape != p._vshape or t.get_device() != device.index
            or not t.is_contiguous()):
        raise ValueError(f"{name} must be a contiguous {p._tdtype} tensor of shape ({p.c},) on {device}")
    return t.data_ptr()


def _params(p, r, y, w_post, gate, w_pre, strides):
    """Checks the operands; the struct of the parameters, and the device.
    strides: the row strides that are not dense, by name."""
    s = _strided(r, p._shape, p._tdtype, None, "r")
    dev = r.device
    if s is not _DENSE[2]:
        strides["r"] = s[0]
    if y is not None:
        s = _strided(y, p._shape, p._tdtype, dev, "y")
        if s is not _DENSE[2]:
            strides["y"] = s[0]
    elif w_post is not None or gate is not None:
        raise ValueError("w_post and gate need y")
    kind, at = GATE_NONE, None
    if gate is not None:
        if gate.dim() == 1:
            kind, at = GATE_CHANNEL, _vector(gate, p, dev, "gate")
        else:
            kind, at = GATE_ROW, gate.data_ptr()
            s = _strided(gate, p._shape, p._tdtype, dev, "gate")
            if s is not _DENSE[2]:
                strides["gate"] = s[0]
    return BlockParams(None if w_post is None else _vector(w_post, p, dev, "w_post"), at,
                       None if w_pre is None else _vector(w_pre, p, dev, "w_pre"), kind, 0), dev


def _ptr(t):
    return None if t is None else t.data_ptr()


def _rows(p, t, name, device, strides):
    """An output of rows: allocated, or the caller's."""
    import torch

    if t is None:
        return torch.empty(p._shape, dtype=p._tdtype, device=device)
    s = _strided(t, p._shape, p._tdtype, device, name)
    if s is not _DENSE[2]:
        strides[name] = s[0]
    _written(t)
    return t


def _struct(strides):
    return ctypes.byref(BlockStrides(**strides)) if strides else None


def _forward(p, r, y, w_post, gate, w_pre, save, z, n, stats, stream):
    import torch

    st = {}
    params, dev = _params(p, r, y, w_post, gate, w_pre, st)
    if (z is not None and y is None) or (n is not None and w_pre is None):
        raise ValueError("z goes with y, and n with w_pre")
    with _on(dev, stream):
        if y is not None:
            z = _rows(p, z, "z", dev, st)
        if w_pre is not None:
            n = _rows(p, n, "n", dev, st)
        if stats is not None:
            if stats.dtype != torch.float32 or stats.shape != (p.rows, 2) or stats.device != dev or not stats.is_contiguous():
                raise ValueError(f"stats must be a contiguous float32 tensor of shape ({p.rows}, 2) on {dev}")
            _written(stats)
        elif save:
            stats = torch.empty((p.rows, 2), dtype=torch.float32, device=dev)
        _check(_lib.cbd_block_forward(p._h, r.data_ptr(), _ptr(y), ctypes.byref(params), _ptr(z), _ptr(n),
                                      _ptr(stats), _struct(st), _handle(stream, dev)), "cbd_block_forward")
    return z, n, stats


def block_forward(p: BlockPlan, r, y=None, w_post=None, gate=None, w_pre=None, save=False, z=None, n=None, stats=None,
                  stream=None):
    """(z, n) on `stream` (default: torch's current one), and with save, or given
    stats, (z, n, stats); outputs are allocated unless given.  z may be r, and n
    y, for a step in place.  stats [T, 2] (f32) is what block_bwd reads."""
    if _any_records((r, y, w_post, gate, w_pre)):
        if z is not None or n is not None or stats is not None:
            raise ValueError("autograd cannot record a call into a given output: an operand requires gradients "
                             "(or has a tangent); leave the outputs out or call under torch.no_grad()")
        if not r.is_cuda:
            raise ValueError("r must be a GPU torch tensor")
        with _on(r.device, stream):
            z, n, stats = _recorder().apply(r, y, w_post, gate, w_pre, p)
    else:
        z, n, stats = _forward(p, r, y, w_post, gate, w_pre, save, z, n, stats, stream)
        save = save or stats is not None
    return (z, n, stats) if save else (z, n)


def _bwd(p, dz, dn, r, y, stats, w_post, gate, w_pre, want, given, workspace, stream):
    """want: which of dr, dy, dw_post, dgate, dw_pre; given: row outputs."""
    import torch

    st = {}
    params, dev = _params(p, r, y, w_post, gate, w_pre, st)
    for name, t in (("dz", dz), ("dn", dn)):
        if t is not None:
            s = _strided(t, p._shape, p._tdtype, dev, name)
            if s is not _DENSE[2]:
                st[name] = s[0]
    if (w_post is not None or w_pre is not None) and (
            stats is None or stats.dtype != torch.float32 or stats.shape != (p.rows, 2) or stats.device != dev
            or not stats.is_contiguous()):
        raise ValueError(f"stats must be a contiguous float32 tensor of shape ({p.rows}, 2) on {dev}")
    want_r, want_y, want_post, want_gate, want_pre = (
        bool(w) and t is not None for w, t in zip(want, (r, y, w_post, gate, w_pre)))
    row_gate = params.gate_kind == GATE_ROW
    with _on(dev, stream):
        dr = _rows(p, given.get("dr"), "dr", dev, st) if want_r else None
        dy = _rows(p, given.get("dy"), "dy", dev, st) if want_y else None
        dgate = dw_post = dw_pre = None
        if want_gate and row_gate:
            dgate, want_gate = _rows(p, given.get("dgate"), "dgate", dev, st), False
        vectors = want_post + want_gate + want_pre
        if vectors:
            new = iter(torch.empty((vectors, p.c), dtype=p._tdw, device=dev).unbind(0))
            dw_post = next(new) if want_post else None
            dgate = next(new) if want_gate else dgate
            dw_pre = next(new) if want_pre else None
        ws_bytes = 0
        if vectors:
            if workspace is None:
                workspace = torch.empty(p._ws, dtype=torch.uint8, device=dev)
            elif not workspace.is_contiguous() or workspace.device != dev:
                raise ValueError(f"workspace must be a contiguous tensor on {dev}")
            else:
                _written(workspace)
            ws_bytes = workspace.numel() * workspace.element_size()
        grads = BlockGrads(_ptr(dr), _ptr(dy), _ptr(dw_post), _ptr(dgate), _ptr(dw_pre))
        _check(_lib.cbd_block_bwd(p._h, _ptr(dz), _ptr(dn), r.data_ptr(), _ptr(y), _ptr(stats), ctypes.byref(params),
                                  ctypes.byref(grads), _struct(st), _ptr(workspace), ws_bytes,
                                  _handle(stream, dev)), "cbd_block_bwd")
    return dr, dy, dw_post, dgate, dw_pre


def block_bwd(p: BlockPlan, dz, dn, r, y=None, stats=None, w_post=None, gate=None, w_pre=None, dr=None, dy=None,
              dgate=None, output_mask=(True, True, True, True, True), workspace=None, stream=None):
    """(dr, dy, dw_post, dgate, dw_pre) from the gradients of z and n (None:
    zeros); None for parts that are not there or that output_mask leaves out.
    dr, dy and a row gate's dgate are allocated unless given; dr may be dz, and
    dy dn.  The vectors' gradients have the plan's dw_dtype."""
    if _any_records((dz, dn, r, y, w_post, gate, w_pre)):
        raise ValueError("block_bwd is not recorded by autograd and an operand requires gradients (or has a "
                         "tangent); call under torch.no_grad()")
    if dgate is not None and (gate is None or gate.dim() == 1):
        raise ValueError("a given dgate goes with a gate of rows")
    if dy is not None and y is None:
        raise ValueError("dy needs y")
    return _bwd(p, dz, dn, r, y, stats, w_post, gate, w_pre, output_mask, dict(dr=dr, dy=dy, dgate=dgate), workspace,
                stream)


@functools.lru_cache(None)
def _recorder():
    import torch

    class BlockNorm(torch.autograd.Function):
        @staticmethod
        def forward(ctx, r, y, w_post, gate, w_pre, p):
            ctx.set_materialize_grads(False)
            z, n, stats = _forward(p, r, y, w_post, gate, w_pre, True, None, None, None, None)
            ctx.plan = p
            ctx.save_for_backward(r, y, w_post, gate, w_pre, stats)
            ctx.mark_non_differentiable(stats)
            return z, n, stats

        @staticmethod
        @torch.autograd.function.once_differentiable
        def backward(ctx, dz, dn, _):
            r, y, w_post, gate, w_pre, stats = ctx.saved_tensors
            if dz is None and dn is None:
                return (None,) * 6
            dz, dn = (None if g is None else g.contiguous() for g in (dz, dn))
            got = _bwd(ctx.plan, dz, dn, r, y, stats, w_post, gate, w_pre, ctx.needs_input_grad[:5], {}, None, None)
            return (*(None if g is None else g.to(t.dtype) for g, t in zip(got, (r, y, w_post, gate, w_pre))), None)

    return BlockNorm


_plans = {}


def block_norm(r, y=None, w_post=None, gate=None, w_pre=None, scale=1.0, eps=1e-6):
    """(z, n) for r [..., C]; differentiable.  y and a gate of rows have r's
    shape."""
    import torch

    if r.dtype not in (torch.float32, torch.bfloat16):
        raise ValueError(f"rows must be float32 or bfloat16, got {r.dtype}")
    if r.dim() < 1:
        raise ValueError("r needs a last dimension")
    shape, c = r.shape, r.shape[-1]
    for name, t in (("y", y), ("gate", gate if gate is not None and gate.dim() > 1 else None)):
        if t is not None and t.shape != shape:
            raise ValueError(f"{name} must have r's shape {tuple(shape)}, got {tuple(t.shape)}")
    rows = r.numel() // c if c else 0
    key = (rows, c, r.dtype, float(scale), float(eps))
    p = _plans.get(key)
    if p is None:
        if len(_plans) >= 1024:  # served batches come in many sizes; a plan is rebuilt in microseconds
            _plans.clear()
        p = _plans[key] = block_plan(rows, c, F32 if r.dtype == torch.float32 else BF16, scale=scale, eps=eps)

    def flat(t):
        return None if t is None else t.reshape(rows, c)

    z, n = block_forward(p, flat(r), flat(y), w_post, gate if gate is None or gate.dim() == 1 else flat(gate), w_pre)
    return None if z is None else z.view(shape), None if n is None else n.view(shape)
