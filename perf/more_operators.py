"""Gated experts, norms around a block and orthogonalised updates, as cases to
be measured.

Five operators over the framework's types (bf16 and f32, f32 or wider sums):

  gated_fwd  h[t] = act(G_e x[t]) * (U_e x[t]), and with save gu[t] = (G_e x[t], U_e x[t]);
             rows sorted by expert, the gate's and the other projection's weights
             side by side in one tensor
  gated_bwd  dgu[t] = (dh * u * act'(g), dh * act(g)) with dh = D_e^T dy[t], the
             gradient that reaches the two projections from behind the block's
             last projection D
  block_fwd  z = r + scale * gate * (norm(y) * w_post),  n = norm(z) * w_pre, and
             with save the two factors 1 / rms of every row
  block_bwd  the gradients of r, y, w_post, gate and w_pre from those of z and n
  ortho      X = M / (|M| + 1e-7), then steps of X = a X + (b A + c A A) X with
             A = X X^T; each matrix of a stack by itself

norm(v) = v / sqrt(mean(v^2) + eps).  `ends[e]` is the row after expert e's
last one; rows past the last end belong to no expert and come out as zeros.
"""
import math
import random

import torch

own = False

_DT = {"bf16": torch.bfloat16, "f32": torch.float32}
_BYTES = {"bf16": 2, "f32": 4}
_EPS = 1e-6
_COEFFICIENTS = (3.4445, -4.7750, 2.0315)


# ---------------------------------------------------------------- cases

def _gated(name, op, tokens, experts, c, k, dtype="bf16", w_layout="ekc", act="silu", save=False,
           skew=0.5, tail=0, gap=0, top=0, route=1):
    """tokens: rows; c: the model's width; k: the block's; tail: of the rows,
    those past the last expert's; skew: spread of the experts' popularity
    (log-normal); gap: extra elements between rows of the row operands (a slice
    of a wider buffer); top: the rows come from tokens that each pick `top`
    different experts (0: independent draws); route: seed of the sizes."""
    return dict(name=name, op=op, tokens=tokens, experts=experts, c=c, k=k, dtype=dtype,
                w_layout=w_layout, act=act, save=save, skew=skew, tail=tail, gap=gap, top=top, route=route)


def _block(name, op, rows, c, dtype="bf16", post=True, gate="channel", save=False, dw="bf16", scale=1.0, gap=0):
    """post: the block's output is normed; gate: "none", "channel" (one vector
    for all rows) or "row" (a tensor like y); dw: type of the vectors' gradients."""
    return dict(name=name, op=op, rows=rows, c=c, dtype=dtype, post=post, gate=gate, save=save, dw=dw,
                scale=scale, gap=gap)


def _ortho(name, matrices, rows, cols, dtype="f32", steps=5):
    return dict(name=name, op="ortho", matrices=matrices, rows=rows, cols=cols, dtype=dtype, steps=steps)


def listed():
    return [
        # One token of a served model that picks 8 of 64 experts: latency.
        _gated("gated-serve-1", "gated_fwd", 8, 64, 2048, 1408, top=8),
        # A served batch of 64 such tokens: every expert's weights, a few rows each.
        _gated("gated-serve-64", "gated_fwd", 512, 64, 2048, 1408, top=8),
        # One micro-batch of training, kept for the backward pass.
        _gated("gated-train", "gated_fwd", 32768, 32, 4096, 2048, save=True, route=2),
        # f32 checking run of a small layer with odd widths, rows inside a wider buffer.
        _gated("gated-odd-f32", "gated_fwd", 3001, 7, 515, 389, dtype="f32", act="gelu", save=True, gap=5, tail=40),
        # The backward pass of an ordinary fine-grained layer.
        _gated("gated-bwd-fine", "gated_bwd", 16384, 64, 2048, 1408, skew=0.8),
        # Widths that no tile divides, output-major weights, a few experts with most rows.
        _gated("gated-bwd-odd", "gated_bwd", 4099, 12, 1000, 776, w_layout="eck", act="gelu", skew=1.0, tail=3),
        # One served token between two blocks: latency.
        _block("block-serve-1", "block_fwd", 1, 4096),
        # One micro-batch of training between two blocks.
        _block("block-train", "block_fwd", 32768, 4096, save=True, scale=0.5),
        # Its backward pass, the vectors' gradients kept in f32.
        _block("block-bwd-train", "block_bwd", 32768, 4096, dw="f32", scale=0.5),
        # f32 checking run of a small block with a gate for every row.
        _block("block-bwd-odd", "block_bwd", 3001, 515, dtype="f32", gate="row", dw="f32", scale=0.25, gap=3),
        # Updates of a small layer of experts.
        _ortho("ortho-small", 16, 256, 512),
        # Updates of a large layer of experts.
        _ortho("ortho-large", 8, 4096, 2048, dtype="bf16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _unnamed(case):
    del case["name"]
    return case


def draw(rng):
    op = rng.choice(["gated_fwd", "gated_fwd", "gated_bwd", "block_fwd", "block_bwd", "ortho"])
    dtype = "f32" if rng.random() < 0.25 else "bf16"
    step = rng.choice([1, 8, 8, 64, 64])
    if op == "ortho":
        rows, cols = (max(step, step * round(_log(rng, 16, 4096) / step)) for _ in range(2))
        small = min(rows, cols)
        most = max(1, int(2.2e11 / (4.0 * small * rows * cols + 2.0 * small ** 3)))
        return _unnamed(_ortho("", _log(rng, 1, min(64, most)), rows, cols, dtype=rng.choice(["bf16", "f32"]),
                               steps=rng.choice([3, 5, 5, 6])))
    if op in ("block_fwd", "block_bwd"):
        c = max(step, step * round(_log(rng, 32, 8192) / step))
        rows = _log(rng, 1, max(2, (60_000_000 if dtype == "f32" else 130_000_000) // c))
        return _unnamed(_block("", op, rows, c, dtype=dtype, post=rng.random() < 0.8,
                               gate=rng.choice(["none", "channel", "row"]),
                               save=op == "block_fwd" and rng.random() < 0.5,
                               dw="f32" if dtype == "f32" else rng.choice(["bf16", "f32"]),
                               scale=rng.choice([1.0, 0.5, 0.1]), gap=rng.choice([0, 0, step])))
    experts = _log(rng, 1, 128)
    c, k = (max(step, step * round(_log(rng, 48, 4096) / step)) for _ in range(2))
    while experts * c * k > 300_000_000:
        experts = max(1, experts // 2)
    products = 2 if op == "gated_fwd" else 1
    cap = 1.0e12 if dtype == "bf16" else 1.0e11
    tokens = _log(rng, 1, max(2, min(60000, int(cap / (2.0 * c * k * products)))))
    return _unnamed(_gated("", op, tokens, experts, c, k, dtype=dtype, w_layout=rng.choice(["ekc", "eck"]),
                           act=rng.choice(["silu", "silu", "gelu", "relu"]),
                           save=op == "gated_fwd" and rng.random() < 0.5, skew=rng.choice([0.0, 0.5, 1.5]),
                           tail=rng.choice([0, 0, min(tokens - 1, 17)]), gap=rng.choice([0, 0, step]),
                           route=rng.randrange(1 << 30)))


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


def _rows(gen, rows, width, gap, dtype, scale):
    t = torch.empty(rows, width + gap, dtype=dtype, device="cuda").normal_(0.0, scale, generator=gen)
    return t[:, :width] if gap else t


def _weights(gen, case, outputs, inputs):
    """[E, outputs, inputs] in the layout "ekc", [E, inputs, outputs] in "eck"."""
    shape = (outputs, inputs) if case["w_layout"] == "ekc" else (inputs, outputs)
    t = torch.empty(case["experts"], *shape, dtype=_DT[case["dtype"]], device="cuda")
    return t.normal_(0.0, inputs ** -0.5, generator=gen)


def _inputs(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    dt = _DT[case["dtype"]]
    if case["op"] == "ortho":
        # A momentum: a few directions that most of it lies in, and noise.
        n, r, c = case["matrices"], case["rows"], case["cols"]
        rank = max(1, min(r, c) // 8)
        left = torch.empty(n, r, rank, device="cuda").normal_(generator=gen)
        right = torch.empty(n, rank, c, device="cuda").normal_(generator=gen)
        noise = torch.empty(n, r, c, device="cuda").normal_(generator=gen)
        return dict(m=(1e-3 * (torch.bmm(left, right) * rank ** -0.5 + 0.3 * noise)).to(dt))
    if case["op"] in ("block_fwd", "block_bwd"):
        T, C, gap = case["rows"], case["c"], case["gap"]
        out = dict(r=_rows(gen, T, C, gap, dt, 2.0), y=_rows(gen, T, C, gap, dt, 0.7))

        def near(mean, spread):
            return torch.empty(C, device="cuda").normal_(mean, spread, generator=gen).to(dt)

        out["w_post"] = near(1.0, 0.2) if case["post"] else None
        out["w_pre"] = near(1.0, 0.2)
        out["gate"] = (None if case["gate"] == "none" else near(0.5, 0.3) if case["gate"] == "channel"
                       else _rows(gen, T, C, gap, dt, 0.5))
        if case["op"] == "block_bwd":
            out["dz"], out["dn"] = _rows(gen, T, C, gap, dt, 0.02), _rows(gen, T, C, gap, dt, 0.02)
            # What the forward pass keeps: 1 / rms of y (1, where it is not normed) and of z.
            parts = []
            for i in range(0, T, 4096):
                s = slice(i, i + 4096)
                y = out["y"][s].double()
                ry = torch.ones_like(y[:, :1])
                v = y
                if case["post"]:
                    ry = torch.rsqrt((y * y).mean(1, keepdim=True) + _EPS)
                    v = y * ry * out["w_post"].double()
                if case["gate"] != "none":
                    v = v * (out["gate"] if case["gate"] == "channel" else out["gate"][s]).double()
                z = out["r"][s].double() + case["scale"] * v
                parts.append(torch.cat([ry, torch.rsqrt((z * z).mean(1, keepdim=True) + _EPS)], 1).float())
            out["stats"] = torch.cat(parts)
        return out
    counts = _counts(case)
    random.Random(seed).shuffle(counts)
    ends, at = [], 0
    for n in counts:
        at += n
        ends.append(at)
    T, C, K, gap = case["tokens"], case["c"], case["k"], case["gap"]
    out = dict(host_ends=ends, ends=torch.tensor(ends, dtype=torch.int32, device="cuda"))
    if case["op"] == "gated_fwd":
        out["x"], out["w"] = _rows(gen, T, C, gap, dt, 1.0), _weights(gen, case, 2 * K, C)
    else:
        out["dy"], out["w"] = _rows(gen, T, C, gap, dt, 0.02), _weights(gen, case, C, K)
        out["gu"] = _rows(gen, T, 2 * K, gap, dt, 1.0)
    return out


def prepare(case, seed):
    state = _inputs(case, seed)
    state["case"] = case
    if own:
        import dnn_conv2d_bwd_amd as cbd

        op = case["op"]
        if op == "ortho":
            state["plan"] = cbd.ortho_plan(case["matrices"], case["rows"], case["cols"], dtype=case["dtype"],
                                           steps=case["steps"])
        elif op in ("block_fwd", "block_bwd"):
            state["plan"] = cbd.block_plan(case["rows"], case["c"], dtype=case["dtype"], dw_dtype=case["dw"],
                                           scale=case["scale"], eps=_EPS)
        else:
            c, k = (case["c"], 2 * case["k"]) if op == "gated_fwd" else (case["k"], case["c"])
            state["plan"] = cbd.expert_plan(case["tokens"], case["experts"], c, k, w_layout=case["w_layout"],
                                            dtype=case["dtype"])
    return state


# ---------------------------------------------------------------- one pass

def _own(s):
    import dnn_conv2d_bwd_amd as cbd

    case, p = s["case"], s["plan"]
    op = case["op"]
    if op == "gated_fwd":
        return cbd.expert_gated_forward(p, s["x"], s["w"], s["ends"], act=case["act"], save=case["save"])
    if op == "gated_bwd":
        return cbd.expert_gated_bwd(p, s["dy"], s["w"], s["gu"], s["ends"], act=case["act"])
    if op == "block_fwd":
        return cbd.block_forward(p, s["r"], s["y"], w_post=s["w_post"], gate=s["gate"], w_pre=s["w_pre"],
                                 save=case["save"])
    if op == "block_bwd":
        return cbd.block_bwd(p, s["dz"], s["dn"], s["r"], s["y"], s["stats"], w_post=s["w_post"],
                             gate=s["gate"], w_pre=s["w_pre"])
    return cbd.orthogonalize(p, s["m"])


_GELU = math.sqrt(2.0 / math.pi)


def _act(name, g):
    """The activation and its derivative."""
    if name == "relu":
        on = (g > 0).to(g.dtype)
        return g * on, on
    if name == "silu":
        s = 1.0 / (1.0 + (-g).exp())
        return g * s, s * (1.0 + g * (1.0 - s))
    t = (_GELU * (g + 0.044715 * g * g * g)).tanh()
    return 0.5 * g * (1.0 + t), 0.5 * (1.0 + t) + 0.5 * g * (1.0 - t * t) * _GELU * (1.0 + 0.134145 * g * g)


def _gated_fwd(s, case):
    T, K, dt = case["tokens"], case["k"], _DT[case["dtype"]]
    h = torch.zeros(T, K, dtype=dt, device="cuda")
    gu = torch.zeros(T, 2 * K, dtype=dt, device="cuda") if case["save"] else None
    lo = 0
    for e, hi in enumerate(s["host_ends"]):
        if hi > lo:
            w = s["w"][e].float()
            both = s["x"][lo:hi].float() @ (w.t() if case["w_layout"] == "ekc" else w)
            h[lo:hi] = _act(case["act"], both[:, :K])[0] * both[:, K:]
            if gu is not None:
                gu[lo:hi] = both
        lo = hi
    return h if gu is None else (h, gu)


def _gated_bwd(s, case):
    T, K = case["tokens"], case["k"]
    dgu = torch.zeros(T, 2 * K, dtype=_DT[case["dtype"]], device="cuda")
    lo = 0
    for e, hi in enumerate(s["host_ends"]):
        if hi > lo:
            w = s["w"][e].float()
            dh = s["dy"][lo:hi].float() @ (w if case["w_layout"] == "ekc" else w.t())
            gu = s["gu"][lo:hi].float()
            a, slope = _act(case["act"], gu[:, :K])
            dgu[lo:hi, :K] = dh * gu[:, K:] * slope
            dgu[lo:hi, K:] = dh * a
        lo = hi
    return dgu


def _block_fwd(s, case):
    dt = _DT[case["dtype"]]
    y = s["y"].float()
    ry = 1.0 / ((y * y).mean(1, keepdim=True) + _EPS).sqrt()
    if case["post"]:
        y = y * ry * s["w_post"].float()
    if s["gate"] is not None:
        y = y * s["gate"].float()
    z = s["r"].float() + case["scale"] * y
    rz = 1.0 / ((z * z).mean(1, keepdim=True) + _EPS).sqrt()
    n = z * rz * s["w_pre"].float()
    if not case["save"]:
        return z.to(dt), n.to(dt)
    if not case["post"]:
        ry = torch.ones_like(ry)
    return z.to(dt), n.to(dt), torch.cat([ry, rz], 1)


def _block_bwd(s, case):
    dt, dw = _DT[case["dtype"]], _DT[case["dw"]]
    y, scale = s["y"].float(), case["scale"]
    ry, rz = s["stats"][:, :1], s["stats"][:, 1:]
    normed = y * ry if case["post"] else y
    a = normed * s["w_post"].float() if case["post"] else y
    gated = a * s["gate"].float() if s["gate"] is not None else a
    zn = (s["r"].float() + scale * gated) * rz
    dn = s["dn"].float()
    # Sums over all rows are in 64 bits.
    dw_pre = (dn * zn).sum(0, dtype=torch.float64)
    v = dn * s["w_pre"].float()
    dz = s["dz"].float() + rz * (v - zn * (v * zn).mean(1, keepdim=True))
    da = scale * dz
    dgate = None
    if s["gate"] is not None:
        dgate = da * a
        dgate = dgate.to(dt) if case["gate"] == "row" else dgate.sum(0, dtype=torch.float64).to(dw)
        da = da * s["gate"].float()
    dy, dw_post = da, None
    if case["post"]:
        dw_post = (da * normed).sum(0, dtype=torch.float64).to(dw)
        v = da * s["w_post"].float()
        dy = ry * (v - normed * (v * normed).mean(1, keepdim=True))
    return dz.to(dt), dy.to(dt), dw_post, dgate, dw_pre.to(dw)


def _newton_schulz(s, case):
    a, b, c = _COEFFICIENTS
    m = s["m"].float()
    tall = case["rows"] > case["cols"]
    norm = s["m"].double().square().sum((1, 2), keepdim=True).sqrt()
    x = m / (norm + 1e-7).float()
    if tall:
        x = x.transpose(1, 2).contiguous()
    for _ in range(case["steps"]):
        xx = torch.bmm(x, x.transpose(1, 2))
        x = a * x + torch.bmm(b * xx + c * torch.bmm(xx, xx), x)
    return (x.transpose(1, 2) if tall else x).to(s["m"].dtype).contiguous()


def run(state):
    if own:
        return _own(state)
    case = state["case"]
    plain = dict(gated_fwd=_gated_fwd, gated_bwd=_gated_bwd, block_fwd=_block_fwd, block_bwd=_block_bwd,
                 ortho=_newton_schulz)
    return plain[case["op"]](state, case)


def work(case):
    op, b = case["op"], _BYTES[case["dtype"]]
    if op == "ortho":
        n, r, c = case["matrices"], case["rows"], case["cols"]
        s = min(r, c)
        # Products of a matrix with its transpose and of A with itself are
        # symmetric: half of each is enough.
        return {"bytes": 2 * n * r * c * b, "flops": n * case["steps"] * (3 * s * r * c + s ** 3)}
    if op in ("block_fwd", "block_bwd"):
        T, C = case["rows"], case["c"]
        row_gate, channel_gate = case["gate"] == "row", case["gate"] == "channel"
        vectors = (1 + case["post"] + channel_gate) * C
        if op == "block_fwd":
            return {"bytes": (4 + row_gate) * T * C * b + vectors * b + 8 * T * case["save"], "flops": 12 * T * C}
        return {"bytes": (6 + 2 * row_gate) * T * C * b + vectors * (b + _BYTES[case["dw"]]) + 8 * T,
                "flops": 30 * T * C}
    T, E, C, K = case["tokens"], case["experts"], case["c"], case["k"]
    rows, busy = T - case["tail"], sum(1 for n in _counts(case) if n)
    if op == "gated_fwd":
        out = T * K * (3 if case["save"] else 1)
        return {"bytes": (rows * C + out + busy * 2 * K * C) * b + 4 * E, "flops": 4 * rows * C * K}
    return {"bytes": (rows * (C + 2 * K) + 2 * T * K + busy * C * K) * b + 4 * E, "flops": 2 * rows * C * K}


# ---------------------------------------------------------------- 64 bits

def _exact_act(name, g):
    if name == "relu":
        return torch.relu(g)
    if name == "silu":
        return g * torch.sigmoid(g)
    return g * torch.sigmoid(2.0 * _GELU * (g + 0.044715 * g ** 3))  # (1 + tanh v) / 2 = sigmoid(2 v)


def _slope(name, g):
    with torch.enable_grad():
        g = g.detach().requires_grad_(True)
        return torch.autograd.grad(_exact_act(name, g).sum(), g)[0]


def exact(case, seed):
    s = _inputs(case, seed)
    f64 = torch.float64
    op = case["op"]
    if op == "ortho":
        a, b, c = _COEFFICIENTS
        outs = []
        for m in s["m"]:
            x = m.to(f64)
            x = x / (torch.linalg.matrix_norm(x) + 1e-7)
            for _ in range(case["steps"]):
                # The polynomial from the smaller side, whichever that is.
                if case["rows"] <= case["cols"]:
                    q = torch.mm(x, x.t())
                    x = torch.mm(torch.addmm(b * q, q, q, alpha=c), x).add_(x, alpha=a)
                else:
                    q = torch.mm(x.t(), x)
                    x = torch.mm(x, torch.addmm(b * q, q, q, alpha=c)).add_(x, alpha=a)
            outs.append(x)
        return torch.stack(outs)
    if op in ("block_fwd", "block_bwd"):
        T, gate = case["rows"], s["gate"]
        named = dict(w_post=s["w_post"], gate=gate if case["gate"] == "channel" else None, w_pre=s["w_pre"])
        total = {k: None if v is None else torch.zeros(v.shape, dtype=f64, device="cuda") for k, v in named.items()}
        parts = []
        for i in range(0, T, 2048):
            at = slice(i, i + 2048)
            grad = op == "block_bwd"
            leaf = {k: None if v is None else v.to(f64).requires_grad_(grad) for k, v in named.items()}
            for k in ("r", "y"):
                leaf[k] = s[k][at].to(f64).requires_grad_(grad)
            if case["gate"] == "row":
                leaf["gate"] = gate[at].to(f64).requires_grad_(grad)
            with torch.set_grad_enabled(grad):
                v = leaf["y"]
                inv_y = torch.ones_like(v[:, :1])
                if case["post"]:
                    inv_y = (v.square().sum(1, keepdim=True) / case["c"] + _EPS).pow(-0.5)
                    v = v * inv_y * leaf["w_post"]
                z = leaf["r"] + (v * case["scale"] if leaf["gate"] is None else v * leaf["gate"] * case["scale"])
                inv_z = (z.square().sum(1, keepdim=True) / case["c"] + _EPS).pow(-0.5)
                n = z * inv_z * leaf["w_pre"]
            if not grad:
                parts.append((z, n, torch.cat([inv_y, inv_z], 1)))
                continue
            want = [k for k, v in leaf.items() if v is not None]
            got = dict(zip(want, torch.autograd.grad([z, n], [leaf[k] for k in want],
                                                     [s["dz"][at].to(f64), s["dn"][at].to(f64)])))
            for k in total:
                if total[k] is not None:
                    total[k] += got[k]
            parts.append((got["r"], got["y"]) + ((got["gate"],) if case["gate"] == "row" else ()))
        whole = [torch.cat(p) for p in zip(*parts)]
        if op == "block_fwd":
            return tuple(whole if case["save"] else whole[:2])
        return whole[0], whole[1], total["w_post"], whole[2] if case["gate"] == "row" else total["gate"], total["w_pre"]
    bounds, K = [0] + s["host_ends"], case["k"]
    spans = [(e, slice(bounds[e], bounds[e + 1])) for e in range(case["experts"]) if bounds[e + 1] > bounds[e]]
    h = torch.zeros(case["tokens"], K, dtype=f64, device="cuda")
    gu = torch.zeros(case["tokens"], 2 * K, dtype=f64, device="cuda")
    # As [E][in][out] (gated_fwd) and [E][out][in] (gated_bwd), whichever way they are stored.
    w = s["w"].transpose(1, 2) if (op == "gated_fwd") == (case["w_layout"] == "ekc") else s["w"]
    for e, at in spans:
        if op == "gated_fwd":
            g, u = (torch.mm(s["x"][at].to(f64), part.to(f64)) for part in w[e].split(K, 1))
            h[at], gu[at] = _exact_act(case["act"], g) * u, torch.cat([g, u], 1)
        else:
            dh = torch.mm(s["dy"][at].to(f64), w[e].to(f64))
            g, u = s["gu"][at].to(f64).split(K, 1)
            gu[at] = torch.cat([dh * u * _slope(case["act"], g), dh * _exact_act(case["act"], g)], 1)
    if op == "gated_bwd":
        return gu
    return (h, gu) if case["save"] else h
