"""Expert layer: products grouped by expert with ragged row counts.

    p = cbd.expert_plan(tokens=t, experts=e, c=c, k=k, dtype="bf16")
    y  = cbd.expert_forward(p, x, w, ends)               # y[t] = W_e x[t]
    dx = cbd.expert_bwd_data(p, dy, w, ends)             # dx[t] = W_e^T dy[t]
    dw = cbd.expert_bwd_weight(p, dy, x, ends)           # dW_e = sum dy[t] x[t]^T

Rows are sorted by expert; `ends[e]` (int32 or int64, on the GPU) is the row
after expert e's last one.  Rows past the last end belong to no expert and
come out as zeros; an expert without rows gets a zero gradient.  W is
[E, K, C] ("ekc") or [E, C, K] ("eck").  Row tensors and weights may be
strided views with a contiguous last dimension.  include/cbd.h states the
operation in full.

Autograd records the three calls where an operand requires gradients; each is
linear in both operands, so their gradients are these calls again, to any
order.  Into a given output nothing can be recorded: such a call is refused,
like torch's with out=.  Forward-mode derivatives are not there and raise.

`expert_linear` and `expert_linear_bwd` build and cache the plan themselves.
"""
from __future__ import annotations

import contextlib
import ctypes
import functools

from . import BF16, F32, _check, _dtype, _lib, _torch_dtype

EKC, ECK = 0, 1
FORWARD, BWD_DATA, BWD_WEIGHT = 0, 1, 2
EXPERT_KERNEL_AUTO, EXPERT_KERNEL_GENERIC, EXPERT_KERNEL_MFMA, EXPERT_KERNEL_STREAM = -1, 0, 1, 2
EXPERT_KERNEL_NAMES = {0: "generic", 1: "mfma", 2: "stream"}


class ExpertProblem(ctypes.Structure):
    _fields_ = [("tokens", ctypes.c_int64), ("experts", ctypes.c_int64), ("c", ctypes.c_int64),
                ("k", ctypes.c_int64), ("w_layout", ctypes.c_int32), ("dtype", ctypes.c_int32),
                ("dw_dtype", ctypes.c_int32), ("ends_bits", ctypes.c_int32)]


class ExpertOptions(ctypes.Structure):
    _fields_ = [("force_kernel", ctypes.c_int32), ("reserved", ctypes.c_int32 * 3)]


class ExpertStrides(ctypes.Structure):
    _fields_ = [("x_row", ctypes.c_int64), ("y_row", ctypes.c_int64), ("w_row", ctypes.c_int64),
                ("w_expert", ctypes.c_int64)]


class ExpertInfo(ctypes.Structure):
    _fields_ = [("kernel", ctypes.c_int32), ("tile_m", ctypes.c_int32), ("tile_n", ctypes.c_int32),
                ("threads", ctypes.c_int32), ("grid", ctypes.c_int64), ("flops", ctypes.c_int64)]


def _bind():
    P = ctypes.POINTER
    V = ctypes.c_void_p
    _lib.cbd_expert_plan.argtypes = [P(ExpertProblem), P(ExpertOptions), P(V)]
    _lib.cbd_expert_plan_destroy.argtypes = [V]
    _lib.cbd_expert_plan_destroy.restype = None
    _lib.cbd_expert_plan_info.argtypes = [V, ctypes.c_int32, P(ExpertInfo)]
    _lib.cbd_expert_forward.argtypes = [V, V, V, V, V, P(ExpertStrides), V]
    _lib.cbd_expert_bwd_data.argtypes = [V, V, V, V, V, P(ExpertStrides), V]
    _lib.cbd_expert_bwd_weight.argtypes = [V, V, V, V, V, ctypes.c_int32, P(ExpertStrides), V]
    for f in ("plan", "plan_info", "forward", "bwd_data", "bwd_weight"):
        getattr(_lib, "cbd_expert_" + f).restype = ctypes.c_int


_bind()


def _w_layout(v):
    if isinstance(v, str):
        return {"ekc": EKC, "eck": ECK}[v.lower()]
    return int(v)


class ExpertPlan:
    """Owns cbd_expert_plan_t objects (one per width of ends); immutable; safe
    to run from several streams."""

    def __init__(self, tokens, experts, c, k, w_layout=EKC, dtype=BF16, dw_dtype=None,
                 force_kernel=EXPERT_KERNEL_AUTO):
        self.tokens, self.experts, self.c, self.k = int(tokens), int(experts), int(c), int(k)
        self.w_layout, self.dtype = _w_layout(w_layout), _dtype(dtype)
        self.dw_dtype = self.dtype if dw_dtype is None else _dtype(dw_dtype)
        self._h = {}
        opt = ExpertOptions(int(force_kernel))
        for bits in (32, 64):
            prob = ExpertProblem(self.tokens, self.experts, self.c, self.k, self.w_layout, self.dtype,
                                 self.dw_dtype, bits)
            h = ctypes.c_void_p()
            _check(_lib.cbd_expert_plan(ctypes.byref(prob), ctypes.byref(opt), ctypes.byref(h)),
                   "cbd_expert_plan")
            self._h[bits] = h
        self.w_shape = ((self.experts, self.k, self.c) if self.w_layout == EKC
                        else (self.experts, self.c, self.k))
        self._tdtype = _torch_dtype(self.dtype)
        self._tdw = _torch_dtype(self.dw_dtype)

    def info(self, op=FORWARD) -> ExpertInfo:
        """What `op` launches on dense, 16-byte aligned tensors."""
        out = ExpertInfo()
        _check(_lib.cbd_expert_plan_info(self._h[32], op, ctypes.byref(out)), "cbd_expert_plan_info")
        return out

    def __del__(self):
        lib = _lib  # None during interpreter shutdown
        for h in getattr(self, "_h", {}).values():
            if lib is not None and h.value:
                lib.cbd_expert_plan_destroy(h)
        self._h = {}


def expert_plan(tokens, experts, c, k, w_layout="ekc", dtype="bf16", dw_dtype=None,
                force_kernel=EXPERT_KERNEL_AUTO) -> ExpertPlan:
    """dw_dtype: type of the weight gradient (default: dtype; "f32" keeps the
    gradients of bf16 operands unrounded)."""
    return ExpertPlan(tokens, experts, c, k, w_layout, dtype, dw_dtype, force_kernel)


_DENSE = {2: (0,), 3: (0, 0)}


def _strided(t, shape, dtype, device, name):
    """Checks a tensor; its strides in elements but the last (0: dense)."""
    if (getattr(t, "dtype", None) is dtype and t.shape == shape and t.is_cuda and t.is_contiguous()
            and (device is None or t.get_device() == device.index)):
        return _DENSE[len(shape)]
    if not hasattr(t, "data_ptr") or not t.is_cuda:
        raise ValueError(f"{name} must be a GPU torch tensor")
    if t.dtype != dtype:
        raise ValueError(f"{name} has dtype {t.dtype}, plan wants {dtype}")
    if tuple(t.shape) != shape:
        raise ValueError(f"{name} must have shape {shape}, got {tuple(t.shape)}")
    if device is not None and t.device != device:
        raise ValueError(f"{name} is on {t.device}, not on {device}")
    st = t.stride()
    if st[-1] != 1 and shape[-1] != 1 and t.numel():
        raise ValueError(f"the last dimension of {name} must be contiguous")
    if t.is_contiguous():
        return _DENSE[len(shape)]
    out = []
    for n, s in zip(shape[:-1], st):
        if n > 1 and s < 1:
            raise ValueError(f"{name} repeats rows (stride {s}); make it contiguous")
        out.append(s if n > 1 else 0)
    return tuple(out)


def _handle(stream, device):
    import torch

    if stream is None:
        # The raw handle: a Stream object costs 2 us, a seventh of a small call.
        return torch._C._cuda_getCurrentRawStream(device.index)
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


_HERE = contextlib.nullcontext()


def _on(device, stream):
    """Context in which outputs are allocated and kernels launched: the
    tensors' device and the call's stream (so that the caching allocator ties
    new memory to the stream that writes it)."""
    import torch

    if stream is None:
        return _HERE if torch.cuda.current_device() == device.index else torch.cuda.device(device)
    if not hasattr(stream, "cuda_stream"):
        stream = torch.cuda.ExternalStream(int(stream), device=device)
    return torch.cuda.stream(stream)


def _written(tensors):
    """Tells autograd that the library writes into tensors of the caller's, so
    that a backward pass that saved one of them refuses the new contents."""
    import torch

    torch.autograd.graph.increment_version(tensors)


def _ends(p, ends, device):
    import torch

    if not hasattr(ends, "data_ptr") or not ends.is_cuda or ends.get_device() != device.index:
        raise ValueError(f"ends must be a tensor on {device}")
    if ends.dtype not in (torch.int32, torch.int64):
        raise ValueError(f"ends must be int32 or int64, got {ends.dtype}")
    if ends.shape != (p.experts,) or not ends.is_contiguous():
        raise ValueError(f"ends must be contiguous with shape ({p.experts},), got {tuple(ends.shape)}")
    return 32 if ends.dtype == torch.int32 else 64


def _strides(x, y, w):
    if x is y is _DENSE[2] and w is _DENSE[3]:
        return None
    return ctypes.byref(ExpertStrides(x[0], y[0], w[1], w[0]))


def _product(p, op, rows, w, ends, out, stream):
    import torch

    fwd = op == FORWARD
    wide_in, wide_out = (p.c, p.k) if fwd else (p.k, p.c)
    in_name, out_name = ("x", "y") if fwd else ("dy", "dx")
    s_in = _strided(rows, (p.tokens, wide_in), p._tdtype, None, in_name)
    dev = rows.device
    s_w = _strided(w, p.w_shape, p._tdtype, dev, "w")
    bits = _ends(p, ends, dev)
    with _on(dev, stream):
        if out is None:
            out, s_out = torch.empty((p.tokens, wide_out), dtype=p._tdtype, device=dev), _DENSE[2]
        else:
            s_out = _strided(out, (p.tokens, wide_out), p._tdtype, dev, out_name)
            _written(out)
        st = _strides(s_in, s_out, s_w) if fwd else _strides(s_out, s_in, s_w)
        f = _lib.cbd_expert_forward if fwd else _lib.cbd_expert_bwd_data
        _check(f(p._h[bits], rows.data_ptr(), w.data_ptr(), ends.data_ptr(), out.data_ptr(), st,
                 _handle(stream, dev)), "cbd_expert_forward" if fwd else "cbd_expert_bwd_data")
    return out


def _weight(p, dy, x, ends, dw, accumulate, stream):
    import torch

    s_y = _strided(dy, (p.tokens, p.k), p._tdtype, None, "dy")
    dev = dy.device
    s_x = _strided(x, (p.tokens, p.c), p._tdtype, dev, "x")
    bits = _ends(p, ends, dev)
    with _on(dev, stream):
        if dw is None:
            dw, s_w = torch.empty(p.w_shape, dtype=p._tdw, device=dev), _DENSE[3]
        else:
            s_w = _strided(dw, p.w_shape, p._tdw, dev, "dw")
            _written(dw)
        _check(_lib.cbd_expert_bwd_weight(p._h[bits], dy.data_ptr(), x.data_ptr(), ends.data_ptr(),
                                          dw.data_ptr(), 1 if accumulate else 0, _strides(s_x, s_y, s_w),
                                          _handle(stream, dev)), "cbd_expert_bwd_weight")
    return dw


def _records(a, b):
    """Whether autograd would record a product of a and b, or carry their
    tangents through it."""
    import torch

    if (getattr(a, "requires_grad", False) or getattr(b, "requires_grad", False)) and torch.is_grad_enabled():
        return True
    forward = torch.autograd.forward_ad
    return forward._current_level >= 0 and any(
        isinstance(t, torch.Tensor) and forward.unpack_dual(t).tangent is not None for t in (a, b))


def _any_records(operands):
    """_records of any number of operands (None: left out)."""
    import torch

    if torch.is_grad_enabled():
        for t in operands:
            if t is not None and getattr(t, "requires_grad", False):
                return True
    return torch.autograd.forward_ad._current_level >= 0 and any(_records(t, None) for t in operands)


@functools.lru_cache(None)
def _recorder():
    import torch

    class ExpertProduct(torch.autograd.Function):
        @staticmethod
        def forward(ctx, p, op, a, b, ends):
            ctx.plan, ctx.op = p, op
            need_a, need_b = ctx.needs_input_grad[2:4]
            ctx.save_for_backward(a if need_b else None, b if need_a else None, ends)
            if op == BWD_WEIGHT:
                return _weight(p, a, b, ends, None, False, None)
            return _product(p, op, a, b, ends, None, None)

        @staticmethod
        def backward(ctx, g):
            p, op = ctx.plan, ctx.op
            a, b, ends = ctx.saved_tensors
            need_a, need_b = ctx.needs_input_grad[2:4]
            # An f32 weight gradient's gradient becomes an operand of the next products.
            g = g.to(p._tdtype).contiguous()
            ga = gb = None
            if op == FORWARD:       # x, w
                ga = expert_bwd_data(p, g, b, ends) if need_a else None
                gb = expert_bwd_weight(p, g, a, ends).to(p._tdtype) if need_b else None
            elif op == BWD_DATA:    # dy, w
                ga = expert_forward(p, g, b, ends) if need_a else None
                gb = expert_bwd_weight(p, a, g, ends).to(p._tdtype) if need_b else None
            else:                   # dy, x
                ga = expert_forward(p, b, g, ends) if need_a else None
                gb = expert_bwd_data(p, a, g, ends) if need_b else None
            return None, None, ga, gb, None

    return ExpertProduct


def _recorded(p, op, a, b, ends, out, stream):
    if out is not None:
        raise ValueError("autograd cannot record a call into a given output: an operand requires gradients "
                         "(or has a tangent); leave the output out or call under torch.no_grad()")
    # The node belongs to the call's stream, so that its backward runs there.
    with _on(a.device, stream) if a.is_cuda else _HERE:
        return _recorder().apply(p, op, a, b, ends)


def expert_forward(p: ExpertPlan, x, w, ends, y=None, stream=None):
    """y[t] = W_e x[t] on `stream` (default: torch's current one); y is
    allocated unless given, and returned."""
    if _records(x, w):
        return _recorded(p, FORWARD, x, w, ends, y, stream)
    return _product(p, FORWARD, x, w, ends, y, stream)


def expert_bwd_data(p: ExpertPlan, dy, w, ends, dx=None, stream=None):
    """dx[t] = W_e^T dy[t]."""
    if _records(dy, w):
        return _recorded(p, BWD_DATA, dy, w, ends, dx, stream)
    return _product(p, BWD_DATA, dy, w, ends, dx, stream)


def expert_bwd_weight(p: ExpertPlan, dy, x, ends, dw=None, accumulate=False, stream=None):
    """dW_e = sum over the rows of e of dy[t] x[t]^T, in the layout of W;
    accumulate: added to the given dw."""
    if accumulate and dw is None:
        raise ValueError("accumulate needs dw")
    if _records(dy, x):
        return _recorded(p, BWD_WEIGHT, dy, x, ends, dw, stream)
    return _weight(p, dy, x, ends, dw, accumulate, stream)


_plans = {}


def _cached(tokens, w_shape, w_layout, tdtype, dw_dtype):
    import torch

    lay = _w_layout(w_layout)
    e, a, b = w_shape
    c, k = (b, a) if lay == EKC else (a, b)
    key = (tokens, e, c, k, lay, tdtype, dw_dtype)
    p = _plans.get(key)
    if p is None:
        if len(_plans) >= 1024:  # served batches come in many sizes; a plan is rebuilt in microseconds
            _plans.clear()
        if tdtype not in (torch.float32, torch.bfloat16):
            raise ValueError(f"operands must be float32 or bfloat16, got {tdtype}")
        p = _plans[key] = expert_plan(tokens, e, c, k, lay, F32 if tdtype == torch.float32 else BF16,
                                      dw_dtype)
    return p


def expert_linear(x, w, ends, w_layout="ekc"):
    """y[t] = W_e x[t] for x [T, C], w [E, K, C] or [E, C, K]; differentiable."""
    p = _cached(x.shape[0], tuple(w.shape), w_layout, w.dtype, None)
    return expert_forward(p, x, w, ends)


def expert_linear_bwd(dy, x, w, ends, w_layout="ekc", output_mask=(True, True), dw_dtype=None):
    """(dx, dw) of expert_linear, each None where the mask leaves it out."""
    p = _cached(x.shape[0], tuple(w.shape), w_layout, w.dtype, dw_dtype)
    dx = expert_bwd_data(p, dy, w, ends) if output_mask[0] else None
    dw = expert_bwd_weight(p, dy, x, ends) if output_mask[1] else None
    return dx, dw
