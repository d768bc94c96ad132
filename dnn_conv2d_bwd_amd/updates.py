"""Orthogonalised updates: Newton-Schulz steps on a stack of matrices.

    p = cbd.ortho_plan(matrices, rows, cols, dtype="f32")
    o = cbd.orthogonalize(p, m)              # m [matrices, rows, cols]
    cbd.orthogonalize(p, m, out=m)           # in place

Every matrix by itself: X = M / (|M| + eps), then `steps` times X = a X + (b A +
c A A) X with A = X X^T, which draws the singular values towards 1 and leaves
the singular vectors; the result times `scale`.  Weights of experts [E, K, C]
are such a stack as they are; matrices and rows may be strided.

`orthogonalized(m)` makes the plan itself.  Nothing is recorded by autograd:
where an operand requires gradients the call is refused (use torch.no_grad()).
A tensor that is written to counts as changed in place.  include/cbd.h states
the operation in full.
"""
from __future__ import annotations

import ctypes

from . import F32, _check, _dtype, _lib, _torch_dtype
from .experts import _any_records, _handle, _on, _strided, _written


class OrthoProblem(ctypes.Structure):
    _fields_ = [("matrices", ctypes.c_int64), ("rows", ctypes.c_int64), ("cols", ctypes.c_int64),
                ("dtype", ctypes.c_int32), ("steps", ctypes.c_int32), ("eps", ctypes.c_double),
                ("scale", ctypes.c_double), ("coefficients", ctypes.POINTER(ctypes.c_double))]


class OrthoStrides(ctypes.Structure):
    _fields_ = [("in_row", ctypes.c_int64), ("in_matrix", ctypes.c_int64), ("out_row", ctypes.c_int64),
                ("out_matrix", ctypes.c_int64)]


class OrthoInfo(ctypes.Structure):
    _fields_ = [("tile_symmetric", ctypes.c_int32), ("tile_step", ctypes.c_int32),
                ("tile_symmetric_rest", ctypes.c_int32), ("tile_step_rest", ctypes.c_int32), ("launches", ctypes.c_int32),
                ("slices", ctypes.c_int32), ("flops", ctypes.c_int64)]


def _bind():
    P = ctypes.POINTER
    V = ctypes.c_void_p
    U = ctypes.c_uint64
    _lib.cbd_ortho_plan.argtypes = [P(OrthoProblem), P(V)]
    _lib.cbd_ortho_plan_destroy.argtypes = [V]
    _lib.cbd_ortho_plan_destroy.restype = None
    _lib.cbd_ortho_plan_info.argtypes = [V, P(OrthoInfo)]
    _lib.cbd_ortho_workspace_size.argtypes = [V, P(U)]
    _lib.cbd_orthogonalize.argtypes = [V, V, V, P(OrthoStrides), V, U, V]
    for f in ("cbd_ortho_plan", "cbd_ortho_plan_info", "cbd_ortho_workspace_size", "cbd_orthogonalize"):
        getattr(_lib, f).restype = ctypes.c_int


_bind()


class OrthoPlan:
    """Owns a cbd_ortho_plan_t; immutable; safe to run from several streams (a
    workspace each)."""

    def __init__(self, matrices, rows, cols, dtype=F32, steps=5, coefficients=None, eps=1e-7, scale=1.0):
        self.matrices, self.rows, self.cols = int(matrices), int(rows), int(cols)
        self.dtype, self.steps = _dtype(dtype), int(steps)
        flat = None
        if coefficients is not None:
            triples = [[float(v) for v in c] for c in coefficients]
            if len(triples) == 1:
                triples *= max(self.steps, 0)
            if len(triples) != self.steps or any(len(c) != 3 for c in triples):
                raise ValueError(f"coefficients must be {self.steps} triples, or one for all steps")
            flat = [v for c in triples for v in c]
            flat = (ctypes.c_double * len(flat))(*flat)
        prob = OrthoProblem(self.matrices, self.rows, self.cols, self.dtype, self.steps, float(eps), float(scale),
                            None if flat is None else ctypes.cast(flat, ctypes.POINTER(ctypes.c_double)))
        h = ctypes.c_void_p()
        _check(_lib.cbd_ortho_plan(ctypes.byref(prob), ctypes.byref(h)), "cbd_ortho_plan")
        self._h = h
        out = ctypes.c_uint64()
        _check(_lib.cbd_ortho_workspace_size(h, ctypes.byref(out)), "cbd_ortho_workspace_size")
        self._ws = int(out.value)
        self._tdtype = _torch_dtype(self.dtype)

    def info(self) -> OrthoInfo:
        """What a call launches."""
        out = OrthoInfo()
        _check(_lib.cbd_ortho_plan_info(self._h, ctypes.byref(out)), "cbd_ortho_plan_info")
        return out

    def workspace_size(self) -> int:
        """Bytes of device workspace a call needs."""
        return self._ws

    def __del__(self):
        h = getattr(self, "_h", None)
        lib = _lib  # None during interpreter shutdown
        if lib is not None and h is not None and h.value:
            lib.cbd_ortho_plan_destroy(h)
            self._h = None


def ortho_plan(matrices, rows, cols, dtype="f32", steps=5, coefficients=None, eps=1e-7, scale=1.0) -> OrthoPlan:
    """coefficients: (a, b, c) of each step, [(a, b, c)] for all; None: (3.4445,
    -4.7750, 2.0315), whose five steps bring singular values above 0.01 of the
    norm to between 0.68 and 1.14."""
    return OrthoPlan(matrices, rows, cols, dtype, steps, coefficients, eps, scale)


def orthogonalize(p: OrthoPlan, m, out=None, workspace=None, stream=None):
    """The orthogonalised matrices on `stream` (default: torch's current one);
    out is allocated unless given, may be m itself, and is returned."""
    import torch

    if _any_records((m,)):
        raise ValueError("orthogonalize is not recorded by autograd and m requires gradients (or has a tangent); "
                         "call under torch.no_grad()")
    shape = (p.matrices, p.rows, p.cols)
    s_in = _strided(m, shape, p._tdtype, None, "m")
    dev = m.device
    with _on(dev, stream):
        if out is None:
            out, s_out = torch.empty(shape, dtype=p._tdtype, device=dev), (0, 0)
        else:
            s_out = _strided(out, shape, p._tdtype, dev, "out")
            _written(out)
        if workspace is None:
            workspace = torch.empty(p._ws, dtype=torch.uint8, device=dev)
        elif not workspace.is_contiguous() or workspace.device != dev:
            raise ValueError(f"workspace must be a contiguous tensor on {dev}")
        else:
            _written(workspace)
        st = OrthoStrides(s_in[1], s_in[0], s_out[1], s_out[0])
        _check(_lib.cbd_orthogonalize(p._h, m.data_ptr(), out.data_ptr(), ctypes.byref(st), workspace.data_ptr(),
                                      workspace.numel() * workspace.element_size(), _handle(stream, dev)),
               "cbd_orthogonalize")
    return out


_plans = {}


def orthogonalized(m, steps=5, coefficients=None, eps=1e-7, scale=1.0):
    """The matrices m [..., rows, cols], orthogonalised, as a new tensor."""
    import torch

    if m.dim() < 2 or m.dtype not in (torch.float32, torch.bfloat16):
        raise ValueError(f"m must be matrices of float32 or bfloat16, got {m.dtype} {tuple(m.shape)}")
    shape = m.shape
    m = m.reshape(-1, *shape[-2:]) if m.dim() != 3 else m
    co = None if coefficients is None else tuple(tuple(float(v) for v in c) for c in coefficients)
    key = (tuple(m.shape), m.dtype, steps, co, eps, scale)
    p = _plans.get(key)
    if p is None:
        if len(_plans) >= 256:
            _plans.clear()
        dtype = "f32" if m.dtype == torch.float32 else "bf16"
        p = _plans[key] = ortho_plan(*m.shape, dtype=dtype, steps=steps, coefficients=co, eps=eps, scale=scale)
    return orthogonalize(p, m).view(shape)
