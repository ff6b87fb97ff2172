"""The operators around a block's products, as a training or serving step calls them.

Three families, each in its plain form (elementary torch operations, 32 bits)
and through the library's calls:

* ``norm_fwd`` / ``norm_bwd``: RMS norm with the residual's addition, with an
  optional e4m3 output in groups of 128 columns, and its backward pass;
* ``expert_fwd`` / ``expert_bwd``: tokens sorted by expert (the plan), copied
  to the experts' order and combined back with the router's weights, and the
  gradients of both copies;
* ``adamw``: one optimizer step over many tensors, its states in 32 or 8 bits.
"""

import math

import torch

own = False

GROUP = 128          # values that share a scale in the 8-bit formats
E4M3_MAX = 448.0
TINY = 2.0 ** -126   # smallest scale: an all-zero group keeps a usable one
EPS = 1e-6

_DT = {"bf16": torch.bfloat16, "f32": torch.float32}
_SIZE = {"bf16": 2, "f32": 4}


# ------------------------------------------------------------------ cases
def listed():
    return [
        # one token through a 70B-wide block's entry: latency
        {"name": "norm_fwd_token", "op": "norm_fwd", "T": 1, "h": 8192, "dtype": "bf16", "residual": True,
         "quantize": False},
        # the 70B block's sequence, with the 8-bit copy beside the bf16 one
        {"name": "norm_fwd_70b_q8", "op": "norm_fwd", "T": 4096, "h": 8192, "dtype": "bf16", "residual": True,
         "quantize": True},
        # a first layer's norm (nothing to add), fp32, ragged
        {"name": "norm_fwd_odd_f32", "op": "norm_fwd", "T": 1021, "h": 1000, "dtype": "f32", "residual": False,
         "quantize": False},
        # the backward of a 16,384-token step, with the residual path's gradient
        {"name": "norm_bwd_16k", "op": "norm_bwd", "T": 16384, "h": 8192, "dtype": "bf16", "residual": True},
        # a short fp32 batch, a width that is no power of two
        {"name": "norm_bwd_odd_f32", "op": "norm_bwd", "T": 333, "h": 4104, "dtype": "f32", "residual": False},
        # a few tokens of a decode step over 8 experts
        {"name": "expert_fwd_small", "op": "expert_fwd", "T": 17, "h": 1024, "k": 2, "experts": 8, "drop": 0.0,
         "dtype": "bf16"},
        # a training step over many small experts
        {"name": "expert_fwd_16k", "op": "expert_fwd", "T": 16384, "h": 4096, "k": 8, "experts": 64, "drop": 0.0,
         "dtype": "bf16"},
        # the backward over few large experts, some assignments over capacity
        {"name": "expert_bwd_drop", "op": "expert_bwd", "T": 4096, "h": 8192, "k": 2, "experts": 8, "drop": 0.1,
         "dtype": "bf16"},
        # fp32, ragged in every direction
        {"name": "expert_bwd_odd_f32", "op": "expert_bwd", "T": 999, "h": 1000, "k": 3, "experts": 60, "drop": 0.05,
         "dtype": "f32"},
        # large bf16 weights with fp32 masters, biases and norms beside them
        {"name": "adamw_32", "op": "adamw", "matrices": 8, "rows": 4096, "cols": 4096, "vectors": 16, "bits": 32,
         "dtype": "bf16", "master": True},
        # the same weights with 8-bit states
        {"name": "adamw_8", "op": "adamw", "matrices": 8, "rows": 4096, "cols": 4096, "vectors": 16, "bits": 8,
         "dtype": "bf16", "master": True},
        # many small tensors of odd sizes: latency
        {"name": "adamw_small", "op": "adamw", "matrices": 40, "rows": 33, "cols": 129, "vectors": 60, "bits": 8,
         "dtype": "f32", "master": False},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm_fwd", "norm_bwd", "expert_fwd", "expert_bwd", "adamw"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if op == "adamw":
        # up to the listed total of 134 million values
        rows, cols = _log(rng, 1, 4096), _log(rng, 16, 4096)
        n = min(_log(rng, 1, 80), max(1, 134_000_000 // (rows * cols)))
        return {"op": op, "matrices": n, "rows": rows, "cols": cols, "vectors": rng.randint(0, 40),
                "bits": rng.choice([8, 32]), "dtype": dtype, "master": dtype == "bf16" and rng.random() < 0.6}
    T, h = _log(rng, 1, 16384), 8 * _log(rng, 8, 1024)
    if op.startswith("norm"):
        T = max(1, min(T, 134_000_000 * 2 // (_SIZE[dtype] * h)))
        case = {"op": op, "T": T, "h": h, "dtype": dtype, "residual": rng.random() < 0.7}
        if op == "norm_fwd":
            case["quantize"] = rng.random() < 0.5
        return case
    k = rng.randint(1, 8)
    T = max(1, min(T, 500_000_000 * 2 // (_SIZE[dtype] * h * k)))
    return {"op": op, "T": T, "h": h, "k": k, "experts": k + _log(rng, 1, 248),
            "drop": rng.choice([0.0, 0.0, 0.1, 0.5]), "dtype": dtype}


# ------------------------------------------------------------------ inputs
def _normal(g, shape, dtype, std=1.0):
    x = torch.empty(shape, dtype=torch.float32, device="cuda")
    return x.normal_(0.0, std, generator=g).to(dtype)


def _to_groups(x):
    """Flat values as rows of GROUP, the last one filled with zeros."""
    n = x.shape[-1]
    x = torch.nn.functional.pad(x, (0, -n % GROUP))
    return x.reshape(*x.shape[:-1], -1, GROUP)


def _quantize(x):
    """e4m3 codes and one fp32 scale per GROUP values of the last dimension."""
    n = x.shape[-1]
    b = _to_groups(x)
    scale = (b.abs().amax(-1) * (1.0 / E4M3_MAX)).clamp_min(TINY)
    q = (b * scale.reciprocal().unsqueeze(-1)).to(torch.float8_e4m3fn)
    return q.reshape(*x.shape[:-1], -1)[..., :n].contiguous(), scale


def _dequantize(q, scale):
    n = q.shape[-1]
    b = _to_groups(q.float()) * scale.unsqueeze(-1)
    return b.reshape(*q.shape[:-1], -1)[..., :n]


def _sort(ids, experts):
    """row [T, k], source [T k] and offsets [experts + 1] of a stable sort by expert; -1 is dropped."""
    flat = ids.reshape(-1).long()
    order = torch.sort(torch.where(flat < 0, experts, flat), stable=True).indices
    counts = torch.bincount(flat + 1, minlength=experts + 1)[1:]
    offsets = torch.zeros(experts + 1, dtype=torch.int64, device=ids.device)
    offsets[1:] = counts.cumsum(0)
    at = torch.arange(flat.numel(), device=ids.device)
    kept = at < offsets[-1]
    row = torch.empty_like(flat)
    row[order] = torch.where(kept, at, -1)
    return {"row": row.int().reshape(ids.shape), "source": torch.where(kept, order, -1).int(),
            "offsets": offsets.int()}


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    dt = _DT[case["dtype"]]
    op = case["op"]
    if op == "norm_fwd" or op == "norm_bwd":
        T, h = case["T"], case["h"]
        s = {"case": case, "X": _normal(g, (T, h), dt), "w": 1.0 + _normal(g, (h,), torch.float32, 0.1), "R": None,
             "dS": None}
        if op == "norm_fwd":
            # the residual stream has grown over the layers before
            s["R"] = _normal(g, (T, h), dt, 4.0) if case["residual"] else None
            return s
        s["dY"] = _normal(g, (T, h), dt)
        s["dS"] = _normal(g, (T, h), dt) if case["residual"] else None
        x = s["X"].float()
        s["rstd"] = torch.rsqrt((x * x).sum(-1) * (1.0 / h) + EPS)
        return s
    if op == "expert_fwd" or op == "expert_bwd":
        T, h, k, E = case["T"], case["h"], case["k"], case["experts"]
        # a router with favourite experts; the weights are its softmax over the chosen ones
        logits = _normal(g, (T, E), torch.float32) + _normal(g, (E,), torch.float32)
        top = logits.topk(k, -1)
        ids = top.indices.int()
        lost = torch.rand((T, k), device="cuda", generator=g) < case["drop"]
        lost |= torch.rand((T, 1), device="cuda", generator=g) < case["drop"] / 8   # whole tokens
        ids = torch.where(lost, -1, ids).int().contiguous()
        s = {"case": case, "ids": ids, "weights": top.values.softmax(-1).contiguous(),
             "Ys": _normal(g, (T * k, h), dt)}
        if op == "expert_fwd":
            s["X"] = _normal(g, (T, h), dt)
        else:
            s["plan"] = _sort(ids, E)
            s["dZ"], s["dXs"] = _normal(g, (T, h), dt), _normal(g, (T * k, h), dt)
        return s
    # a step in the middle of a run: moments as the gradients before have left them. The tensors of a kind lie in
    # one buffer, as a program that writes checkpoints keeps them
    shapes = _shapes(case)
    types = [dt if len(shape) == 2 else torch.float32 for shape in shapes]   # biases and norms stay in fp32
    held = [d == torch.bfloat16 and case["master"] for d in types]
    s = {"case": case, "step": 100, "decay": [0.1 if len(shape) == 2 else 0.0 for shape in shapes]}
    values, p = _buffer(shapes)
    values.normal_(0.0, 0.02, generator=g)
    s["weights"], weights = _buffer([x for x, d in zip(shapes, types) if d != torch.float32], torch.bfloat16)
    s["weights"].copy_(values[:s["weights"].numel()])   # the matrices come first
    s["grads16"], grads16 = _buffer([x for x, d in zip(shapes, types) if d != torch.float32], torch.bfloat16)
    s["grads16"].normal_(0.0, 1e-3, generator=g)
    s["grads32"], grads32 = _buffer([x for x, d in zip(shapes, types) if d == torch.float32])
    s["grads32"].normal_(0.0, 1e-3, generator=g)
    s["values"] = values
    s["params"] = weights + p[len(weights):]
    s["masters"] = [x if h else None for x, h in zip(p, held)]
    s["grads"] = grads16 + grads32
    m, mv = _buffer(shapes)
    m.normal_(0.0, 3e-4, generator=g)
    v, vv = _buffer(shapes)
    v.normal_(0.0, 1e-3, generator=g).square_().add_(1e-9)
    if case["bits"] == 32:
        s["state"] = {"m": m, "v": v}
        s["states"] = [{"m": x, "v": y} for x, y in zip(mv, vv)]
        return s
    s["state"], views = {}, {}
    scales = [(-(-math.prod(shape) // GROUP),) for shape in shapes]
    for name, x in (("m", mv), ("r", [y.sqrt() for y in vv])):
        s["state"][name + "_q"], views[name + "_q"] = _buffer(shapes, torch.float8_e4m3fn)
        s["state"][name + "_scale"], views[name + "_scale"] = _buffer(scales)
        for val, q, scale in zip(x, views[name + "_q"], views[name + "_scale"]):
            codes, sc = _quantize(val.reshape(-1))
            q.copy_(codes.reshape(q.shape))
            scale.copy_(sc)
    s["states"] = [{k: x[i] for k, x in views.items()} for i in range(len(shapes))]
    return s


def _shapes(case):
    return [(case["rows"], case["cols"])] * case["matrices"] + [(case["cols"] + i % 3,) for i in range(case["vectors"])]


def _buffer(shapes, dtype=torch.float32):
    """One zeroed buffer and a view of each shape in it, each view's start on 64 values."""
    at = [0]
    for shape in shapes:
        at.append(at[-1] + -(-math.prod(shape) // 64) * 64)
    flat = torch.zeros(at[-1], dtype=dtype, device="cuda")
    return flat, [flat[i:i + math.prod(shape)].view(shape) for i, shape in zip(at, shapes)]


# ------------------------------------------------------------------ one pass
LR, BETA1, BETA2, ADAM_EPS, GRAD_SCALE = 1e-3, 0.9, 0.999, 1e-8, 0.5


def run(s):
    if own:
        return _run_own(s)
    return {"norm_fwd": _norm_fwd, "norm_bwd": _norm_bwd, "expert_fwd": _expert_fwd, "expert_bwd": _expert_bwd,
            "adamw": _adamw}[s["case"]["op"]](s)


def _run_own(s):
    import vocab_ce_gb300 as tp

    c = s["case"]
    if c["op"] == "norm_fwd":
        return tp.tp_rmsnorm_forward(s["X"], s["w"], R=s["R"], eps=EPS, quantize=c["quantize"])
    if c["op"] == "norm_bwd":
        return tp.tp_rmsnorm_backward(s["dY"], s["X"], s["w"], s["rstd"], dS=s["dS"])
    if c["op"] == "expert_fwd":
        plan = tp.tp_expert_plan(s["ids"], c["experts"])
        return {**plan, "Xs": tp.tp_expert_dispatch_forward(s["X"], plan),
                "Z": tp.tp_expert_combine_forward(s["Ys"], plan, s["weights"])}
    if c["op"] == "expert_bwd":
        grads = tp.tp_expert_combine_backward(s["dZ"], s["Ys"], s["plan"], s["weights"])
        return {**grads, "dX": tp.tp_expert_dispatch_backward(s["dXs"], s["plan"])}
    tp.adamw_step(s["params"], s["grads"], s["states"], lr=LR, step=s["step"], beta1=BETA1, beta2=BETA2,
                  eps=ADAM_EPS, weight_decay=s["decay"], grad_scale=GRAD_SCALE, masters=s["masters"])
    return _updated(s)


def _norm_fwd(s):
    X, R, w = s["X"], s["R"], s["w"]
    out = {}
    S = X
    if R is not None:
        # the stream is held in its own type: what is normalised is what the next layer adds to
        S = out["S"] = (X.float() + R.float()).to(X.dtype)
    x = S.float()
    rstd = torch.rsqrt((x * x).sum(-1) * (1.0 / x.shape[-1]) + EPS)
    y = x * rstd.unsqueeze(-1) * w
    out["Y"], out["rstd"] = y.to(X.dtype), rstd
    if s["case"]["quantize"]:
        out["Q"], out["Q_scale"] = _quantize(y)
    return out


def _norm_bwd(s):
    dy, w, rstd = s["dY"].float(), s["w"], s["rstd"].unsqueeze(-1)
    xh = s["X"].float() * rstd
    g = dy * w
    c = (g * xh).sum(-1, keepdim=True) * (1.0 / g.shape[-1])
    dx = (g - xh * c) * rstd
    if s["dS"] is not None:
        dx = dx + s["dS"].float()
    return {"dX": dx.to(s["X"].dtype), "dw": (dy * xh).sum(0)}


def _gather_sum(rows, row, weights):
    """sum_j weights[t, j] rows[row[t, j]] in 32 bits; -1 adds nothing."""
    x = rows[row.clamp_min(0).long()].float()
    x = torch.where((row >= 0).unsqueeze(-1), x, 0.0)
    return (x if weights is None else x * weights.unsqueeze(-1)).sum(1)


def _expert_fwd(s):
    X, k = s["X"], s["case"]["k"]
    plan = _sort(s["ids"], s["case"]["experts"])
    source = plan["source"]
    Xs = X[torch.div(source.clamp_min(0), k, rounding_mode="floor").long()]
    Xs = torch.where((source >= 0).unsqueeze(-1), Xs, 0.0)
    return {**plan, "Xs": Xs, "Z": _gather_sum(s["Ys"], plan["row"], s["weights"]).to(X.dtype)}


def _expert_bwd(s):
    plan, dZ, Ys = s["plan"], s["dZ"], s["Ys"]
    T, k = plan["row"].shape
    source = plan["source"]
    kept = (source >= 0).unsqueeze(-1)
    at = source.clamp_min(0).long()
    dz = dZ[torch.div(at, k, rounding_mode="floor")].float()
    dYs = torch.where(kept, dz * s["weights"].reshape(-1)[at].unsqueeze(-1), 0.0).to(dZ.dtype)
    dots = (torch.where(kept, Ys.float(), 0.0) * dz).sum(-1)
    row = plan["row"].reshape(-1)
    dweights = torch.where(row >= 0, dots[row.clamp_min(0).long()], 0.0).reshape(T, k)
    return {"dYs": dYs, "dweights": dweights, "dX": _gather_sum(s["dXs"], plan["row"], None).to(dZ.dtype)}


def _adamw(s):
    bc1, bc2 = 1.0 - BETA1 ** s["step"], 1.0 - BETA2 ** s["step"]
    for p, master, grad, st, wd in zip(s["params"], s["masters"], s["grads"], s["states"], s["decay"]):
        g = grad.float() * GRAD_SCALE
        if "m" in st:
            m, v = st["m"], st["v"]
        else:
            m = _dequantize(st["m_q"].reshape(-1), st["m_scale"]).reshape(p.shape)
            v = _dequantize(st["r_q"].reshape(-1), st["r_scale"]).reshape(p.shape)
            v = v * v
        m = m * BETA1 + g * (1.0 - BETA1)
        v = v * BETA2 + (g * g) * (1.0 - BETA2)
        r = v.sqrt()
        x = (p if master is None else master).float()
        x = x * (1.0 - LR * wd) - (m / (r * (1.0 / math.sqrt(bc2)) + ADAM_EPS)) * (LR / bc1)
        if master is not None:
            master.copy_(x)
        p.copy_(x)
        if "m" in st:
            st["m"].copy_(m)
            st["v"].copy_(v)
        else:
            for name, new in (("m", m), ("r", r)):
                q, scale = _quantize(new.reshape(-1))
                st[name + "_q"].copy_(q.reshape(p.shape))
                st[name + "_scale"].copy_(scale)
    return _updated(s)


def _updated(s):
    """The step's tensors, whole: `values` holds the fp32 parameters and the masters."""
    return {"weights": s["weights"], "values": s["values"], **s["state"]}


# ------------------------------------------------------------------ what a pass cannot do without
def work(case):
    op, e = case["op"], _SIZE[case["dtype"]]
    if op == "norm_fwd":
        n = case["T"] * case["h"]
        b = n * e * (4 if case["residual"] else 2) + 4 * case["h"] + 4 * case["T"]
        if case["quantize"]:
            b += n + 4 * case["T"] * (-(-case["h"] // GROUP))
        return {"bytes": b, "flops": 6 * n}
    if op == "norm_bwd":
        n = case["T"] * case["h"]
        return {"bytes": n * e * (4 if case["residual"] else 3) + 8 * case["h"] + 4 * case["T"], "flops": 11 * n}
    if op == "expert_fwd" or op == "expert_bwd":
        T, k, h = case["T"], case["k"], case["h"]
        kept = T * k * (1.0 - case["drop"]) * (1.0 - case["drop"] / 8)
        rows, one = kept * h * e, T * h * e
        if op == "expert_fwd":
            # the plan, X once, the experts' rows written, their results read, Z
            return {"bytes": 2 * one + rows + T * k * h * e + 16 * T * k, "flops": 2 * kept * h}
        # dZ, Ys and dXs read, dYs and dX written
        return {"bytes": 2 * one + 2 * rows + T * k * h * e + 12 * T * k, "flops": 4 * kept * h}
    n2, n1 = case["matrices"] * case["rows"] * case["cols"], sum(case["cols"] + i % 3 for i in range(case["vectors"]))
    state = 16 if case["bits"] == 32 else 4 + 16.0 / GROUP
    each = 3 * e + (8 - e if case["master"] else 0)   # with a master the weight itself is only written
    return {"bytes": n2 * (each + state) + n1 * (12 + state), "flops": 14 * (n1 + n2)}


# ------------------------------------------------------------------ the definitions in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    d = torch.float64
    op = case["op"]
    if op == "norm_fwd" or op == "norm_bwd":
        x = s["X"].to(d)
        if op == "norm_fwd":
            out = {}
            if s["R"] is not None:
                out["S"] = (x + s["R"].to(d)).to(s["X"].dtype)
                x = out["S"].to(d)
            rstd = x.pow(2).mean(-1).add(EPS).pow(-0.5)
            y = x * rstd[:, None] * s["w"].to(d)
            out["Y"], out["rstd"] = y, rstd
            if case["quantize"]:
                # the values that the codes stand for, before their rounding
                b = _to_groups(y)
                out["Q_scale"] = b.abs().amax(-1).div(E4M3_MAX).clamp_min(TINY)
                q = (b / out["Q_scale"][..., None]).reshape(y.shape[0], -1)
                out["Q"] = q[:, :y.shape[1]]
            return out
        rstd = x.pow(2).mean(-1, keepdim=True).add(EPS).pow(-0.5)
        dy, n = s["dY"].to(d), x.shape[1]
        gw = dy * s["w"].to(d)
        dx = rstd * gw - rstd.pow(3) * x * torch.einsum("th,th->t", gw, x)[:, None] / n
        if s["dS"] is not None:
            dx += s["dS"].to(d)
        return {"dX": dx, "dw": torch.einsum("th,th->h", dy, x * rstd)}
    if op == "expert_fwd" or op == "expert_bwd":
        T, k, E, h = case["T"], case["k"], case["experts"], case["h"]
        ids = s["ids"].reshape(-1).long()
        # every expert's assignments in order, one expert after the other
        at = torch.cat([torch.nonzero(ids == e).reshape(-1) for e in range(E)])
        n = at.numel()
        w = torch.zeros(T * k, dtype=d, device="cuda")
        w[:n] = s["weights"].reshape(-1).to(d)[at]
        token = at // k
        if op == "expert_fwd":
            X = torch.zeros((T * k, h), dtype=d, device="cuda")
            X[:n] = s["X"].to(d)[token]
            Z = torch.zeros((T, h), dtype=d, device="cuda").index_add_(0, token, s["Ys"][:n].to(d) * w[:n, None])
            row = torch.full((T * k,), -1, device="cuda")
            row[at] = torch.arange(n, device="cuda")
            source = torch.full((T * k,), -1, device="cuda")
            source[:n] = at
            edge = torch.tensor([0] + [int((ids == e).sum()) for e in range(E)], device="cuda").cumsum(0)
            return {"row": row.reshape(T, k), "source": source, "offsets": edge, "Xs": X, "Z": Z}
        dz = s["dZ"].to(d)[token]
        dY = torch.zeros((T * k, h), dtype=d, device="cuda")
        dY[:n] = dz * w[:n, None]
        dw = torch.zeros(T * k, dtype=d, device="cuda")
        dw[at] = torch.einsum("nh,nh->n", dz, s["Ys"][:n].to(d))
        dX = torch.zeros((T, h), dtype=d, device="cuda").index_add_(0, token, s["dXs"][:n].to(d))
        return {"dYs": dY, "dweights": dw.reshape(T, k), "dX": dX}
    out = {}
    for name, buf in _updated(s).items():
        out[name] = buf.to(d)   # every tensor's part is written below
    flat = {name: buf.data_ptr() for name, buf in _updated(s).items()}

    def put(name, view, val):
        i = (view.data_ptr() - flat[name]) // view.element_size()
        out[name][i:i + view.numel()] = val.reshape(-1)

    for p, master, grad, st, wd in zip(s["params"], s["masters"], s["grads"], s["states"], s["decay"]):
        g = grad.to(d) * GRAD_SCALE
        if "m" in st:
            m, v = st["m"].to(d), st["v"].to(d)
        else:
            n = p.numel()
            m, v = (st[a].reshape(-1).to(d) * st[b].to(d).repeat_interleave(GROUP)[:n]
                    for a, b in (("m_q", "m_scale"), ("r_q", "r_scale")))
            m, v = m.reshape(p.shape), v.reshape(p.shape).pow(2)
        m = torch.lerp(g, m, BETA1)
        v = torch.lerp(g * g, v, BETA2)
        mh, vh = m / (1 - BETA1 ** s["step"]), v / (1 - BETA2 ** s["step"])
        x = (p if master is None else master).to(d)
        x = x - LR * (mh / (vh.sqrt() + ADAM_EPS) + wd * x)
        if p.dtype == torch.bfloat16:
            put("weights", p, x)
        if p.dtype == torch.float32 or master is not None:
            put("values", p if master is None else master, x)
        if "m" in st:
            put("m", st["m"], m)
            put("v", st["v"], v)
            continue
        for name, val in (("m", m), ("r", v.sqrt())):
            # the values that the codes stand for, before their rounding
            b = _to_groups(val.reshape(-1))
            scale = b.abs().amax(-1).div(E4M3_MAX).clamp_min(TINY)
            put(name + "_scale", st[name + "_scale"], scale)
            put(name + "_q", st[name + "_q"], (b / scale[:, None]).reshape(-1)[:val.numel()])
    return out
