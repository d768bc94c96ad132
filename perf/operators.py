"""Expert-layer products and gradient clipping, as cases to be measured.

Five operators over the framework's types (bf16 and f32, f32 or wider sums):

  forward     y[t]  = W_e x[t]            rows sorted by expert, e = e(t)
  bwd_data    dx[t] = W_e^T dy[t]
  bwd_weight  dW_e  = sum over the rows t of expert e of dy[t] x[t]^T
  grad_norm   sqrt of the sum of squares over a list of tensors
  clip        the list scaled by min(1, max_norm / (norm + 1e-6)), and the norm

`ends[e]` is the row after expert e's last one; rows past the last end belong
to no expert and come out as zeros.  Weights are [E][K][C] ("ekc") or
[E][C][K] ("eck") for C inputs and K outputs.
"""
import math
import random

import torch

own = False

_DT = {"bf16": torch.bfloat16, "f32": torch.float32}
_BYTES = {"bf16": 2, "f32": 4}


# ---------------------------------------------------------------- cases

def _expert(name, op, tokens, experts, c, k, dtype="bf16", w_layout="ekc", dw="bf16", skew=0.5,
            tail=0, gap=0, top=0, route=1):
    """tokens: rows of x and y; tail: of them, rows past the last expert's;
    skew: spread of the experts' popularity (log-normal); gap: extra elements
    between rows of the row operands (a slice of a wider buffer); top: the rows
    come from tokens that each pick `top` different experts (0: independent
    draws); route: seed of the experts' sizes."""
    return dict(name=name, op=op, tokens=tokens, experts=experts, c=c, k=k, dtype=dtype,
                w_layout=w_layout, dw=dw, skew=skew, tail=tail, gap=gap, top=top, route=route)


def _grads(name, op, tensors, total, mix, max_norm=1.0, shift=0, route=1):
    """A list of `tensors` gradients of `total` elements together, log-normal
    sizes; mix: share of f32 tensors (the others are bf16); shift: elements by
    which every second tensor's start is off the allocation's alignment."""
    return dict(name=name, op=op, tensors=tensors, total=total, mix=mix, max_norm=max_norm,
                shift=shift, route=route)


def listed():
    return [
        # One token of a served model that picks 8 of 64 experts: latency.
        _expert("serve-1", "forward", 8, 64, 2048, 1408, top=8),
        # A served batch of 64 such tokens: every expert's weights, a few rows each.
        _expert("serve-64", "forward", 512, 64, 2048, 1408, top=8),
        # One micro-batch of training, the largest product.
        _expert("train-fwd", "forward", 65536, 32, 4096, 2048, route=2),
        # f32 checking run of a small layer with odd widths, rows inside a wider buffer.
        _expert("odd-fwd-f32", "forward", 3001, 7, 515, 389, dtype="f32", gap=5, tail=40),
        # The backward pass of an ordinary fine-grained layer.
        _expert("fine-bwd-data", "bwd_data", 16384, 64, 2048, 1408, skew=0.8),
        # Widths that no tile divides, input-major weights.
        _expert("odd-bwd-data", "bwd_data", 4099, 12, 1000, 776, w_layout="eck", skew=1.0),
        # Weight gradients of the large layer, kept in f32.
        _expert("train-bwd-weight", "bwd_weight", 65536, 32, 4096, 2048, dw="f32", route=2),
        # Weight gradients of a small layer, some experts with hardly a row.
        _expert("odd-bwd-weight", "bwd_weight", 5003, 16, 1000, 520, skew=1.5, tail=3),
        # A small network's gradients: latency.
        _grads("norm-small", "grad_norm", 12, 60_000, 1.0),
        # A large model's gradients on one card.
        _grads("norm-large", "grad_norm", 290, 1_500_000_000, 0.1),
        # An ordinary model's mixed list, in flat buffers.
        _grads("clip-mixed", "clip", 60, 120_000_000, 0.4, shift=1),
        # f32 gradients of a layer of experts.
        _grads("clip-large", "clip", 9, 540_000_000, 1.0),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["forward", "forward", "bwd_data", "bwd_weight", "grad_norm", "clip"])
    route = rng.randrange(1 << 30)
    if op in ("grad_norm", "clip"):
        tensors = _log(rng, 1, 400 if op == "grad_norm" else 60)
        total = _log(rng, max(tensors, 1000), 500_000_000)
        return {k: v for k, v in _grads("", op, tensors, total, rng.choice([0.0, 0.3, 1.0]),
                                        max_norm=rng.choice([0.5, 1.0, 1e6]),
                                        shift=rng.choice([0, 0, 1, 3]), route=route).items() if k != "name"}
    dtype = "f32" if rng.random() < 0.2 else "bf16"
    experts = _log(rng, 1, 128)
    step = rng.choice([1, 8, 8, 64, 64])
    c, k = (max(step, step * round(_log(rng, 48, 4096) / step)) for _ in range(2))
    cap = 1.0e12 if dtype == "bf16" else 1.0e11
    top_tokens = max(2, min(60000, int(cap / (2.0 * c * k))))
    tokens = _log(rng, 1, top_tokens)
    while experts * c * k > 400_000_000:
        experts = max(1, experts // 2)
    case = _expert("", op, tokens, experts, c, k, dtype=dtype, w_layout=rng.choice(["ekc", "eck"]),
                   dw="f32" if dtype == "f32" else rng.choice(["bf16", "f32"]),
                   skew=rng.choice([0.0, 0.5, 1.5]), tail=rng.choice([0, 0, min(tokens - 1, 17)]),
                   gap=rng.choice([0, 0, step]), route=route)
    del case["name"]
    return case


# ---------------------------------------------------------------- inputs

def _counts(case):
    """Rows of each expert, as many as `experts`; from the case alone."""
    rng = random.Random(case["route"])
    n, rows = case["experts"], case["tokens"] - case["tail"]
    weight = [math.exp(rng.gauss(0.0, case["skew"])) for _ in range(n)]
    counts = [0] * n
    if case["top"]:
        for _ in range(rows // case["top"]):
            keys = sorted(range(n), key=lambda e: -math.log(rng.random() + 1e-300) / weight[e])
            for e in keys[:case["top"]]:
                counts[e] += 1
    else:
        for e in rng.choices(range(n), weight, k=rows):
            counts[e] += 1
    return counts


def _sizes(case):
    """Elements and type of every gradient; from the case alone."""
    rng = random.Random(case["route"])
    n = case["tensors"]
    weight = [math.exp(rng.gauss(0.0, 1.0)) for _ in range(n)]
    total = sum(weight)
    sizes = [max(1, int(case["total"] * w / total)) for w in weight]
    types = ["f32" if (i + 0.5) / n < case["mix"] else "bf16" for i in range(n)]
    rng.shuffle(types)
    return sizes, types


def _rows(gen, rows, width, gap, dtype, scale):
    t = torch.empty(rows, width + gap, dtype=dtype, device="cuda").normal_(0.0, scale, generator=gen)
    return t[:, :width] if gap else t


def _inputs(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    if case["op"] in ("grad_norm", "clip"):
        sizes, types = _sizes(case)
        host = random.Random(seed)
        grads = []
        for i, (n, ty) in enumerate(zip(sizes, types)):
            off = case["shift"] if i % 2 else 0
            t = torch.empty(n + off, dtype=_DT[ty], device="cuda")
            t.normal_(0.0, math.exp(host.gauss(-6.0, 1.0)), generator=gen)
            grads.append(t[off:])
        return dict(grads=grads)
    counts = _counts(case)
    random.Random(seed).shuffle(counts)
    ends, at = [], 0
    for n in counts:
        at += n
        ends.append(at)
    dt = _DT[case["dtype"]]
    T, E, C, K = case["tokens"], case["experts"], case["c"], case["k"]
    out = dict(host_ends=ends, ends=torch.tensor(ends, dtype=torch.int32, device="cuda"))
    if case["op"] != "bwd_data":
        out["x"] = _rows(gen, T, C, case["gap"], dt, 1.0)
    if case["op"] != "forward":
        out["dy"] = _rows(gen, T, K, case["gap"], dt, 0.02)
    if case["op"] != "bwd_weight":
        shape = (E, K, C) if case["w_layout"] == "ekc" else (E, C, K)
        out["w"] = torch.empty(shape, dtype=dt, device="cuda").normal_(0.0, C ** -0.5, generator=gen)
    return out


def prepare(case, seed):
    state = _inputs(case, seed)
    state["case"] = case
    if own:
        import dnn_conv2d_bwd_amd as cbd

        if case["op"] in ("grad_norm", "clip"):
            state["plan"] = cbd.grad_plan(state["grads"])
        else:
            state["plan"] = cbd.expert_plan(tokens=case["tokens"], experts=case["experts"], c=case["c"],
                                            k=case["k"], w_layout=case["w_layout"], dtype=case["dtype"],
                                            dw_dtype=case["dw"] if case["op"] == "bwd_weight" else None)
    return state


# ---------------------------------------------------------------- one pass

def _own(s):
    import dnn_conv2d_bwd_amd as cbd

    op, p = s["case"]["op"], s["plan"]
    if op == "forward":
        return cbd.expert_forward(p, s["x"], s["w"], s["ends"])
    if op == "bwd_data":
        return cbd.expert_bwd_data(p, s["dy"], s["w"], s["ends"])
    if op == "bwd_weight":
        return cbd.expert_bwd_weight(p, s["dy"], s["x"], s["ends"])
    if op == "grad_norm":
        return cbd.grad_norm(p, s["grads"])
    norm, outs = cbd.clip_grads(p, s["grads"], s["case"]["max_norm"], out=True)
    return [norm, *outs]


def _square_sum(grads):
    """Sum of squares in 64 bits (1e9 terms are too many for 32), in pieces."""
    total = torch.zeros((), dtype=torch.float64, device="cuda")
    for g in grads:
        for part in g.split(1 << 27):
            d = part.double()
            total = total + (d * d).sum()
    return total


def run(state):
    if own:
        return _own(state)
    case = state["case"]
    op = case["op"]
    if op == "grad_norm":
        return _square_sum(state["grads"]).sqrt().float()
    if op == "clip":
        norm = _square_sum(state["grads"]).sqrt()
        scale = (case["max_norm"] / (norm + 1e-6)).clamp(max=1.0)
        return [norm.float()] + [(g.float() * scale.float()).to(g.dtype) for g in state["grads"]]
    T, E, C, K = case["tokens"], case["experts"], case["c"], case["k"]
    ends, lo = state["host_ends"], 0
    dt = _DT[case["dtype"]]
    if op == "bwd_weight":
        dw = torch.zeros((E, K, C) if case["w_layout"] == "ekc" else (E, C, K),
                         dtype=_DT[case["dw"]], device="cuda")
        for e, hi in enumerate(ends):
            if hi > lo:
                x, dy = state["x"][lo:hi].float(), state["dy"][lo:hi].float()
                dw[e] = dy.t() @ x if case["w_layout"] == "ekc" else x.t() @ dy
            lo = hi
        return dw
    rows, wide = (state["x"], K) if op == "forward" else (state["dy"], C)
    out = torch.zeros(T, wide, dtype=dt, device="cuda")
    contracts_last = (op == "forward") == (case["w_layout"] == "ekc")
    for e, hi in enumerate(ends):
        if hi > lo:
            w = state["w"][e].float()
            out[lo:hi] = rows[lo:hi].float() @ (w.t() if contracts_last else w)
        lo = hi
    return out


def work(case):
    if case["op"] in ("grad_norm", "clip"):
        sizes, types = _sizes(case)
        read = sum(n * _BYTES[t] for n, t in zip(sizes, types))
        n = sum(sizes)
        if case["op"] == "grad_norm":
            return {"bytes": read + 4, "flops": 2 * n}
        return {"bytes": 2 * read + 4, "flops": 3 * n}
    T, E, C, K = case["tokens"], case["experts"], case["c"], case["k"]
    b = _BYTES[case["dtype"]]
    rows = T - case["tail"]
    flops = 2 * rows * C * K
    if case["op"] == "bwd_weight":
        return {"bytes": rows * (C + K) * b + E * C * K * _BYTES[case["dw"]] + 4 * E, "flops": flops}
    busy = sum(1 for n in _counts(case) if n)
    read, write = (C, K) if case["op"] == "forward" else (K, C)
    return {"bytes": rows * read * b + T * write * b + busy * C * K * b + 4 * E, "flops": flops}


# ---------------------------------------------------------------- 64 bits

def exact(case, seed):
    s = _inputs(case, seed)
    f64 = torch.float64
    if case["op"] in ("grad_norm", "clip"):
        parts = []
        for g in s["grads"]:
            for i in range(0, g.numel(), 1 << 27):
                v = g[i:i + (1 << 27)].to(f64)
                parts.append(torch.linalg.vector_norm(v).square())
        norm = torch.stack(parts).sum().sqrt()
        if case["op"] == "grad_norm":
            return norm
        by = min(1.0, case["max_norm"] / (float(norm) + 1e-6))
        return [norm] + [g.to(f64).mul_(by) for g in s["grads"]]
    T, E = case["tokens"], case["experts"]
    bounds = [0] + s["host_ends"]
    spans = [(e, slice(bounds[e], bounds[e + 1])) for e in range(E)]
    if case["op"] == "bwd_weight":
        left, right = (s["dy"], s["x"]) if case["w_layout"] == "ekc" else (s["x"], s["dy"])
        return torch.stack([torch.mm(left[rows].to(f64).t(), right[rows].to(f64)) for _, rows in spans])
    src = s["x"] if case["op"] == "forward" else s["dy"]
    # As [E][contracted][produced], whichever way the weights are stored.
    w = s["w"].transpose(1, 2) if (case["op"] == "forward") == (case["w_layout"] == "ekc") else s["w"]
    out = torch.cat([torch.mm(src[rows].to(f64), w[e].to(f64)) for e, rows in spans])
    return torch.cat([out, out.new_zeros(T - bounds[-1], out.shape[1])])
