"""The two ends that a transformer's step has beside its products: the embedding and the attention core.

Two families, each in its plain form (elementary torch operations, 32 bits) and
through the library's calls:

* ``embed_fwd`` / ``embed_bwd``: rows of the token table by id, scaled, and the
  table's gradient, written whole or added to the one that a tied table has
  from the loss;
* ``attn_fwd`` / ``attn_bwd``: causal attention on the fused Q, K, V of packed
  sequences with grouped heads; with a window a query sees the last ``window``
  keys up to its own and the first ``sinks`` of its sequence.
"""

import math

import torch

own = False

_DT = {"bf16": torch.bfloat16, "f32": torch.float32}
_SIZE = {"bf16": 2, "f32": 4}


# ------------------------------------------------------------------ cases
def listed():
    return [
        # the token that a generating model has just chosen: latency
        {"name": "embed_fwd_token", "op": "embed_fwd", "T": 1, "h": 8192, "v": 128256, "dtype": "bf16",
         "scaled": False, "pad": 0.0},
        # a training step's tokens through a 129,024-row table, scaled by the root of the width
        {"name": "embed_fwd_16k", "op": "embed_fwd", "T": 16384, "h": 8192, "v": 128256, "dtype": "bf16",
         "scaled": True, "pad": 0.0},
        # the tied table of the same step: added to the gradient that the loss has written
        {"name": "embed_bwd_tied", "op": "embed_bwd", "T": 16384, "h": 8192, "v": 128256, "dtype": "bf16",
         "scaled": True, "pad": 0.0, "add": True},
        # an untied table of 51,200 rows, all of it written, with padding among the tokens
        {"name": "embed_bwd_whole", "op": "embed_bwd", "T": 8192, "h": 4096, "v": 50257, "dtype": "bf16",
         "scaled": False, "pad": 0.1, "add": False},
        # fp32, ragged, a short batch
        {"name": "embed_bwd_odd_f32", "op": "embed_bwd", "T": 999, "h": 1000, "v": 30001, "dtype": "f32",
         "scaled": True, "pad": 0.05, "add": False},
        # a prompt of a few tokens: latency
        {"name": "attn_fwd_prompt", "op": "attn_fwd", "lengths": "17", "behind": 0, "n_kv": 8, "group": 8, "d": 128,
         "window": 0, "sinks": 0, "dtype": "bf16"},
        # a 70B block's heads on one sequence, every key before the query visible
        {"name": "attn_fwd_70b", "op": "attn_fwd", "lengths": "8192", "behind": 0, "n_kv": 8, "group": 8, "d": 128,
         "window": 0, "sinks": 0, "dtype": "bf16"},
        # two long documents with a window of 1024 and four first tokens kept
        {"name": "attn_fwd_window", "op": "attn_fwd", "lengths": "11000 5350", "behind": 34, "n_kv": 8, "group": 8,
         "d": 128, "window": 1024, "sinks": 4, "dtype": "bf16"},
        # fp32, ragged sequences, a head width that is no power of two
        {"name": "attn_fwd_odd_f32", "op": "attn_fwd", "lengths": "333 1 700", "behind": 3, "n_kv": 2, "group": 3,
         "d": 80, "window": 100, "sinks": 5, "dtype": "f32"},
        # the backward of the 70B block's heads
        {"name": "attn_bwd_70b", "op": "attn_bwd", "lengths": "4096", "behind": 0, "n_kv": 8, "group": 8, "d": 128,
         "window": 0, "sinks": 0, "dtype": "bf16"},
        # the windowed backward over ragged sequences, 32 heads of 96 that share nothing
        {"name": "attn_bwd_window", "op": "attn_bwd", "lengths": "6001 1 900 1290", "behind": 0, "n_kv": 32, "group": 1,
         "d": 96, "window": 512, "sinks": 16, "dtype": "bf16"},
        # fp32, short and ragged
        {"name": "attn_bwd_odd_f32", "op": "attn_bwd", "lengths": "129 400", "behind": 7, "n_kv": 2, "group": 2,
         "d": 64, "window": 0, "sinks": 0, "dtype": "f32"},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["embed_fwd", "embed_bwd", "attn_fwd", "attn_bwd"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if op.startswith("embed"):
        h = 8 * _log(rng, 8, 1024)
        add = rng.random() < 0.5
        # a table of the listed one's bytes at most, of the listed untied one's where all of it is written
        most = 420_000_000 if op == "embed_bwd" and not add else 2_100_000_000
        v = max(128, min(_log(rng, 1000, 128256), most // (_SIZE[dtype] * h)))
        case = {"op": op, "T": _log(rng, 1, 16384), "h": h, "v": v, "dtype": dtype, "scaled": rng.random() < 0.5,
                "pad": rng.choice([0.0, 0.0, 0.05, 0.5])}
        if op == "embed_bwd":
            case["add"] = add
        return case
    n_kv, group = rng.choice([1, 2, 4, 8, 8, 32]), rng.choice([1, 1, 2, 3, 4, 8])
    n_kv = min(n_kv, 64 // group)
    d = rng.choice([128, 128, 64, 96, 80, 8 * rng.randint(2, 16)])
    lengths = [_log(rng, 1, 8192) for _ in range(rng.choice([1, 1, 2, 3, 8]))]
    window = rng.choice([0, 0, _log(rng, 1, 4096)])
    sinks = rng.choice([0, 4, _log(rng, 1, 300)]) if window else 0
    case = {"op": op, "lengths": "", "behind": rng.choice([0, 0, rng.randint(1, 200)]), "n_kv": n_kv, "group": group,
            "d": d, "window": window, "sinks": sinks, "dtype": dtype}
    # visible pairs of all heads as in the listed cases: the largest is 8192 keys over 64 heads
    most = 2_100_000_000 if dtype == "bf16" else 60_000_000
    if op == "attn_bwd":
        most //= 3
    while True:
        case["lengths"] = " ".join(str(n) for n in lengths)
        if sum(_pairs(case)) * n_kv * group <= most:
            return case
        lengths = [max(1, n * 3 // 4) for n in lengths]


def _lengths(case):
    return [int(n) for n in case["lengths"].split()]


def _pairs(case):
    """The pairs of query and visible key of each sequence."""
    out = []
    for n in _lengths(case):
        total = n * (n + 1) // 2
        w, sinks = case["window"], case["sinks"]
        if w and n > w:
            hidden = n - w                                 # of the last query; one less for each before it
            # without sinks 1 + .. + hidden pairs are lost; a query that hides m keys sees min(m, sinks) of them again
            total -= hidden * (hidden + 1) // 2
            s = min(sinks, hidden)
            total += s * (s + 1) // 2 + s * (hidden - s)
        out.append(total)
    return out


# ------------------------------------------------------------------ inputs
def _normal(g, shape, dtype, std=1.0):
    x = torch.empty(shape, dtype=torch.float32, device="cuda")
    return x.normal_(0.0, std, generator=g).to(dtype)


def _padded(v):
    return -(-v // 128) * 128


def _scale(case):
    return math.sqrt(case["h"]) if case["scaled"] else 1.0


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    dt = _DT[case["dtype"]]
    if case["op"].startswith("embed"):
        T, h, v = case["T"], case["h"], case["v"]
        # words by Zipf's law: the share of the id k is log((k + 2) / (k + 1)) / log(v + 1)
        u = torch.rand(T, device="cuda", dtype=torch.float64, generator=g)
        ids = ((v + 1.0) ** u).floor().clamp_(1, v).int() - 1
        ids = torch.where(torch.rand(T, device="cuda", generator=g) < case["pad"], -1, ids).int().contiguous()
        s = {"case": case, "ids": ids}
        if case["op"] == "embed_fwd":
            s["E"] = _normal(g, (_padded(v), h), dt, 0.02)
            return s
        s["dX"] = _normal(g, (T, h), dt)
        if case["add"]:
            # what the loss has left in the tied table's gradient
            s["dE"] = _normal(g, (_padded(v), h), dt, 2.0)
        return s
    n_q, n_kv, d = case["n_kv"] * case["group"], case["n_kv"], case["d"]
    T = sum(_lengths(case)) + case["behind"]
    edges = [0]
    for n in _lengths(case):
        edges.append(edges[-1] + n)
    s = {"case": case, "edges": edges, "offsets": torch.tensor(edges, dtype=torch.int32, device="cuda"),
         "QKV": _normal(g, (T, (n_q + 2 * n_kv) * d), dt)}
    if case["op"] == "attn_bwd":
        s["dO"] = _normal(g, (T, n_q * d), dt)
        s.update(_attn_fwd(s))          # the forward's results, kept for the backward
    return s


# ------------------------------------------------------------------ one pass
def run(s):
    if own:
        return _run_own(s)
    return {"embed_fwd": _embed_fwd, "embed_bwd": _embed_bwd, "attn_fwd": _attn_fwd, "attn_bwd": _attn_bwd}[
        s["case"]["op"]](s)


def _run_own(s):
    import vocab_ce_gb300 as tp

    c = s["case"]
    if c["op"] == "embed_fwd":
        return {"X": tp.tp_embedding_forward(s["ids"], s["E"], v_valid=c["v"], scale=_scale(c))}
    if c["op"] == "embed_bwd":
        return {"dE": tp.tp_embedding_backward(s["dX"], s["ids"], _padded(c["v"]), v_valid=c["v"], scale=_scale(c),
                                               out=s["dE"] if c["add"] else None, accumulate=c["add"])}
    heads = dict(n_heads=c["n_kv"] * c["group"], n_kv_heads=c["n_kv"], offsets=s["offsets"], window=c["window"],
                 sinks=c["sinks"])
    if c["op"] == "attn_fwd":
        return tp.tp_attn_core_forward(s["QKV"], **heads)
    return {"dQKV": tp.tp_attn_core_backward(s["dO"], s["QKV"], s["O"], s["lse"], **heads)}


def _embed_fwd(s):
    ids, E = s["ids"], s["E"]
    x = E[ids.clamp_min(0).long()].float() * _scale(s["case"])
    return {"X": torch.where((ids >= 0).unsqueeze(-1), x, 0.0).to(E.dtype)}


def _embed_bwd(s):
    ids, dX, c = s["ids"], s["dX"], s["case"]
    v_pad = _padded(c["v"])
    at = torch.where(ids < 0, v_pad, ids).long()     # padding goes to a row of its own
    G = torch.zeros((v_pad + 1, c["h"]), device="cuda").index_add_(0, at, dX.float())
    if not c["add"]:
        return {"dE": (G[:v_pad] * _scale(c)).to(dX.dtype)}
    dE = s["dE"]
    at = ids.clamp_min(0).long()
    # a token that is padding writes the row of the id 0 as that row's own tokens do
    dE[at] = (dE[at].float() + G[at] * _scale(c)).to(dE.dtype)
    return {"dE": dE}


def _heads(QKV, c):
    """Q [T, n_kv, group, d], K and V [T, n_kv, d] in 32 bits."""
    x = QKV.float().reshape(QKV.shape[0], c["n_kv"], c["group"] + 2, c["d"])
    return x[:, :, :c["group"]], x[:, :, c["group"]], x[:, :, c["group"] + 1]


def _blocks(s):
    """Query rows of a sequence and the keys that any of them sees, as rows, with the mask."""
    c = s["case"]
    w, sinks = c["window"], c["sinks"]
    for a, b in zip(s["edges"], s["edges"][1:]):
        n = b - a
        rows = max(64, min(1024, (1 << 27) // max(1, c["n_kv"] * c["group"] * n)))
        for q0 in range(0, n, rows):
            q1 = min(n, q0 + rows)
            lo = max(0, q0 - w + 1) if w else 0
            i = torch.arange(q0, q1, device="cuda").unsqueeze(1)
            j = torch.arange(lo, q1, device="cuda")
            first = min(sinks, lo)
            if first:
                j = torch.cat([torch.arange(first, device="cuda"), j])
            seen = j <= i
            if w:
                seen &= (j > i - w) | (j < sinks)
            yield slice(a + q0, a + q1), a + j, seen


def _scores(q, k, seen, c):
    x = torch.einsum("qngd,knd->ngqk", q, k) * (1.0 / math.sqrt(c["d"]))
    return x.masked_fill_(~seen, -math.inf)


def _attn_fwd(s):
    c = s["case"]
    T, n_q = s["QKV"].shape[0], c["n_kv"] * c["group"]
    Q, K, V = _heads(s["QKV"], c)
    O = torch.zeros((T, c["n_kv"], c["group"], c["d"]), device="cuda")
    lse = torch.zeros((n_q, T), device="cuda")
    for rows, keys, seen in _blocks(s):
        x = _scores(Q[rows], K[keys], seen, c)
        m = x.amax(-1, keepdim=True)
        p = torch.exp(x.sub_(m))
        total = p.sum(-1, keepdim=True)
        O[rows] = torch.einsum("ngqk,knd->qngd", p.div_(total), V[keys])
        lse[:, rows] = (m + total.log()).reshape(n_q, -1)
    return {"O": O.reshape(T, n_q * c["d"]).to(s["QKV"].dtype), "lse": lse}


def _attn_bwd(s):
    c = s["case"]
    T = s["QKV"].shape[0]
    Q, K, V = _heads(s["QKV"], c)
    dO = s["dO"].float().reshape(Q.shape)
    delta = (dO * s["O"].float().reshape(Q.shape)).sum(-1)
    lse = s["lse"].reshape(c["n_kv"], c["group"], T)
    grad = torch.zeros((T, c["n_kv"], c["group"] + 2, c["d"]), device="cuda")
    dQ, dK, dV = grad[:, :, :c["group"]], grad[:, :, c["group"]], grad[:, :, c["group"] + 1]
    scale = 1.0 / math.sqrt(c["d"])
    for rows, keys, seen in _blocks(s):
        p = _scores(Q[rows], K[keys], seen, c).sub_(lse[:, :, rows].unsqueeze(-1)).exp_()
        # no key is named twice within a block
        dV[keys] += torch.einsum("ngqk,qngd->knd", p, dO[rows])
        dp = torch.einsum("qngd,knd->ngqk", dO[rows], V[keys])
        ds = dp.sub_(delta[rows].permute(1, 2, 0).unsqueeze(-1)).mul_(p).mul_(scale)
        dQ[rows] = torch.einsum("ngqk,knd->qngd", ds, K[keys])
        dK[keys] += torch.einsum("ngqk,qngd->knd", ds, Q[rows])
    return {"dQKV": grad.reshape(T, -1).to(s["QKV"].dtype)}


# ------------------------------------------------------------------ what a pass cannot do without
def _expected_rows(case):
    """Table rows that the batch's ids name, on average."""
    v, n = case["v"], case["T"] * (1.0 - case["pad"])
    k = torch.arange(1, v + 1, dtype=torch.float64)
    share = torch.log1p(1.0 / k) / math.log(v + 1.0)
    return float((1.0 - (1.0 - share) ** n).sum())


def work(case):
    e = _SIZE[case["dtype"]]
    if case["op"].startswith("embed"):
        T, h = case["T"], case["h"]
        kept, named = T * (1.0 - case["pad"]), _expected_rows(case)
        if case["op"] == "embed_fwd":
            return {"bytes": 4 * T + (named + T) * h * e, "flops": kept * h}
        table = 2 * named if case["add"] else _padded(case["v"])
        return {"bytes": 4 * T + (kept + table) * h * e, "flops": kept * h}
    n_q, n_kv, d = case["n_kv"] * case["group"], case["n_kv"], case["d"]
    T = sum(_lengths(case)) + case["behind"]
    pairs = sum(_pairs(case)) * n_q
    qkv, o, lse = T * (n_q + 2 * n_kv) * d * e, T * n_q * d * e, 4 * T * n_q
    if case["op"] == "attn_fwd":
        return {"bytes": qkv + o + lse, "flops": 4 * d * pairs}
    return {"bytes": 2 * qkv + 2 * o + lse, "flops": 10 * d * pairs}


# ------------------------------------------------------------------ the definitions in 64 bits
def exact(case, seed):
    D = torch.float64
    if case["op"].startswith("attn"):
        # three times the work of the listed cases would take too long here
        cells = sum(n * n for n in _lengths(case)) * case["n_kv"] * case["group"]
        if cells > 16e9:
            return None
    s = prepare(case, seed)
    if case["op"] == "embed_fwd":
        x = torch.zeros((case["T"], case["h"]), dtype=D, device="cuda")
        kept = s["ids"] >= 0
        x[kept] = s["E"][s["ids"][kept].long()].to(D) * _scale(case)
        return {"X": x}
    if case["op"] == "embed_bwd":
        dE = s["dE"].to(D) if case["add"] else torch.zeros((_padded(case["v"]), case["h"]), dtype=D, device="cuda")
        kept = torch.nonzero(s["ids"] >= 0).reshape(-1)
        ids, order = s["ids"][kept].long().sort(stable=True)
        # runs of equal ids as differences of running sums over slices of the columns
        last = torch.ones_like(ids, dtype=torch.bool)
        last[:-1] = ids[1:] != ids[:-1]
        for c0 in range(0, case["h"], 1024):
            total = s["dX"][kept[order], c0:c0 + 1024].to(D).cumsum(0)[last]
            total[1:] -= total[:-1].clone()
            dE[ids[last], c0:c0 + 1024] += total * _scale(case)
        return {"dE": dE}
    n_kv, G, d = case["n_kv"], case["group"], case["d"]
    T = s["QKV"].shape[0]
    x = s["QKV"].reshape(T, n_kv, G + 2, d)
    O = torch.zeros((T, n_kv, G, d), dtype=D, device="cuda")
    lse = torch.zeros((n_kv, G, T), dtype=D, device="cuda")
    grad = torch.zeros((T, n_kv, G + 2, d), dtype=D, device="cuda")
    backward = case["op"] == "attn_bwd"
    for a, b in zip(s["edges"], s["edges"][1:]):
        for n in range(n_kv):
            k, v = x[a:b, n, G].to(D), x[a:b, n, G + 1].to(D)
            for h in range(G):
                for q0 in range(a, b, 2048):
                    q1 = min(b, q0 + 2048)
                    at = torch.arange(q0 - a, q1 - a, device="cuda")[:, None] - torch.arange(q1 - a, device="cuda")
                    hidden = at < 0
                    if case["window"]:
                        old = at >= case["window"]
                        old[:, :case["sinks"]] = False
                        hidden |= old
                    q, kk, vv = x[q0:q1, n, h].to(D), k[:q1 - a], v[:q1 - a]
                    score = torch.mm(q, kk.T) / d ** 0.5
                    score.masked_fill_(hidden, -math.inf)
                    lse[n, h, q0:q1] = torch.logsumexp(score, -1)
                    p = torch.softmax(score, -1)
                    if not backward:
                        O[q0:q1, n, h] = p @ vv
                        continue
                    do = s["dO"].reshape(T, n_kv, G, d)[q0:q1, n, h].to(D)
                    # the softmax's Jacobian, diag(p) - p p^T, on dO V^T
                    g = do @ vv.T
                    g = p * g - p * (p * g).sum(-1, keepdim=True)
                    grad[q0:q1, n, h] = g @ kk / d ** 0.5
                    grad[a:q1, n, G] += g.T @ q / d ** 0.5
                    grad[a:q1, n, G + 1] += p.T @ do
    if backward:
        return {"dQKV": grad.reshape(T, -1)}
    return {"O": O.reshape(T, -1), "lse": lse.reshape(n_kv * G, T)}
