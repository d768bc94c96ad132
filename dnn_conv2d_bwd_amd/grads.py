"""The global gradient norm over a list of tensors, and clipping by it.

    p = cbd.grad_plan(grads)                 # sizes and types of the list
    n = cbd.grad_norm(p, grads)              # f32 scalar tensor on the GPU
    n = cbd.clip_grads(p, grads, 1.0)        # in place; returns the norm
    n, outs = cbd.clip_grads(p, grads, 1.0, out=True)

`clip_grad_norm(grads, max_norm)` makes the plan itself.  f32 and bf16
tensors may be mixed; each must be dense (any order of its dimensions).  The
norm stays on the GPU: nothing here waits for it.  Nothing is recorded by
autograd; tensors that are written to count as changed in place.  include/cbd.h states the
operation in full.
"""
from __future__ import annotations

import ctypes

from . import BF16, F32, _check, _lib
from .experts import _handle, _on, _written


def _bind():
    P = ctypes.POINTER
    V = ctypes.c_void_p
    U = ctypes.c_uint64
    _lib.cbd_grad_plan.argtypes = [P(ctypes.c_int64), P(ctypes.c_int32), ctypes.c_int32, P(V)]
    _lib.cbd_grad_plan_destroy.argtypes = [V]
    _lib.cbd_grad_plan_destroy.restype = None
    _lib.cbd_grad_workspace_size.argtypes = [V, P(U)]
    _lib.cbd_grad_norm.argtypes = [V, P(V), V, V, U, V]
    _lib.cbd_grad_clip.argtypes = [V, P(V), P(V), ctypes.c_double, V, V, U, V]
    for f in ("plan", "workspace_size", "norm", "clip"):
        getattr(_lib, "cbd_grad_" + f).restype = ctypes.c_int


_bind()


def _types():
    import torch

    return {torch.float32: F32, torch.bfloat16: BF16}


class GradPlan:
    """Owns a cbd_grad_plan_t for a list of element counts and types;
    immutable; safe to run from several streams (a workspace each)."""

    def __init__(self, counts, dtypes):
        self.counts = tuple(int(c) for c in counts)
        self.dtypes = tuple(int(d) for d in dtypes)
        if len(self.counts) != len(self.dtypes):
            raise ValueError("counts and dtypes differ in length")
        n = len(self.counts)
        self.list_type = ctypes.c_void_p * max(1, n)
        h = ctypes.c_void_p()
        _check(_lib.cbd_grad_plan((ctypes.c_int64 * max(1, n))(*self.counts),
                                  (ctypes.c_int32 * max(1, n))(*self.dtypes), n, ctypes.byref(h)),
               "cbd_grad_plan")
        self._h = h
        out = ctypes.c_uint64()
        _check(_lib.cbd_grad_workspace_size(h, ctypes.byref(out)), "cbd_grad_workspace_size")
        self._ws = int(out.value)
        import torch

        self._tdtypes = tuple(torch.float32 if d == F32 else torch.bfloat16 for d in self.dtypes)

    def workspace_size(self) -> int:
        """Bytes of device workspace a call needs."""
        return self._ws

    def __del__(self):
        h = getattr(self, "_h", None)
        lib = _lib  # None during interpreter shutdown
        if lib is not None and h is not None and h.value:
            lib.cbd_grad_plan_destroy(h)
            self._h = None


def grad_plan(grads) -> GradPlan:
    """Plan for tensors of these sizes and types (their addresses are not kept)."""
    grads, types = list(grads), _types()
    for i, g in enumerate(grads):
        if g.dtype not in types:
            raise ValueError(f"gradient {i} has dtype {g.dtype}; float32 and bfloat16 are supported")
    return GradPlan([g.numel() for g in grads], [types[g.dtype] for g in grads])


def _dense(t):
    """Whether t's elements fill one block of memory, in any order."""
    if t.is_contiguous():
        return True
    n = 1
    for s, d in sorted((s, d) for s, d in zip(t.stride(), t.shape) if d != 1):
        if s != n:
            return False
        n *= d
    return True


def _pointers(p, tensors, name, device):
    if len(tensors) != len(p.counts):
        raise ValueError(f"{len(tensors)} {name}, the plan is for {len(p.counts)}")
    index = device.index
    for i, (t, n, dt) in enumerate(zip(tensors, p.counts, p._tdtypes)):
        if t.dtype is not dt or t.numel() != n:
            raise ValueError(f"{name} {i} has {t.numel()} elements of {t.dtype}, the plan is for {n} of {dt}")
        if t.get_device() != index:
            raise ValueError(f"{name} {i} is on {t.device}, not on the GPU {device}")
        if not t.is_contiguous() and not _dense(t):
            raise ValueError(f"{name} {i} is not dense in memory")
    return p.list_type(*[t.data_ptr() for t in tensors])


def _device(grads, norm, workspace):
    import torch

    for t in (*grads[:1], norm, workspace):
        if t is not None:
            if t.device.type != "cuda":
                raise ValueError("gradients, norm and workspace must be GPU tensors")
            return t.device
    return torch.device("cuda", torch.cuda.current_device())


def _scratch(p, norm, workspace, device):
    import torch

    if norm is None:
        norm = torch.empty((), dtype=torch.float32, device=device)
    elif norm.dtype != torch.float32 or norm.numel() != 1 or norm.device != device:
        raise ValueError(f"norm must be one float32 on {device}")
    else:
        _written(norm)
    if workspace is None:
        workspace = torch.empty(p._ws, dtype=torch.uint8, device=device)
    elif not workspace.is_contiguous() or workspace.device != device:
        raise ValueError(f"workspace must be a contiguous tensor on {device}")
    else:
        _written(workspace)
    return norm, workspace


def grad_norm(p: GradPlan, grads, norm=None, workspace=None, stream=None):
    """The 2-norm of all elements of all tensors, as an f32 scalar on the GPU."""
    dev = _device(grads, norm, workspace)
    ptrs = _pointers(p, grads, "gradient", dev)
    with _on(dev, stream):
        norm, ws = _scratch(p, norm, workspace, dev)
        _check(_lib.cbd_grad_norm(p._h, ptrs, norm.data_ptr(), ws.data_ptr(),
                                  ws.numel() * ws.element_size(), _handle(stream, dev)), "cbd_grad_norm")
    return norm


def clip_grads(p: GradPlan, grads, max_norm, out=None, norm=None, workspace=None, stream=None):
    """Scales the tensors by min(1, max_norm / (norm + 1e-6)).  out: None, in
    place, returns the norm; True, into new tensors, or a list, into those:
    returns (norm, outs).  New tensors have the layout of their gradient;
    given ones must have its strides."""
    import torch

    dev = _device(grads, norm, workspace)
    ptrs = _pointers(p, grads, "gradient", dev)
    with _on(dev, stream):
        norm, ws = _scratch(p, norm, workspace, dev)
        optrs = None
        if out is True:
            out = [torch.empty_like(g) for g in grads]
            optrs = p.list_type(*[o.data_ptr() for o in out])
        elif out is not None:
            optrs = _pointers(p, out, "output", dev)
            for i, (g, o) in enumerate(zip(grads, out)):
                if g.shape != o.shape or (g.stride() != o.stride() and not (g.is_contiguous() and o.is_contiguous())):
                    raise ValueError(f"output {i} is laid out unlike its gradient")
            _written(out)
        else:
            _written(grads)
        _check(_lib.cbd_grad_clip(p._h, ptrs, optrs, float(max_norm), norm.data_ptr(), ws.data_ptr(),
                                  ws.numel() * ws.element_size(), _handle(stream, dev)), "cbd_grad_clip")
    return norm if out is None else (norm, out)


_plans = {}


def clip_grad_norm(grads, max_norm):
    """Clips the tensors in place and returns their norm before it."""
    grads = list(grads)
    key = tuple((g.numel(), g.dtype) for g in grads)
    p = _plans.get(key)
    if p is None:
        if len(_plans) >= 64:
            _plans.clear()
        p = _plans[key] = grad_plan(grads)
    return clip_grads(p, grads, max_norm)
