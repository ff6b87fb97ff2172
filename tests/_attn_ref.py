"""The attention core in 64 bits, with what a kernel's results may be off by.

U[dtype] is a stored value's half step. A dot of d products in fp32 is off by at
most d 2^-24 times the sum of the products' absolute values; 2^x and the products
around it by a few 2^-24 of the value, and by the error of x. In bf16 the factors
P and dS of the second products are rounded too, by U each, relative to their value.

All of this is relative, and ends where a type's normal numbers do: below 2^-126, in
bf16 as in fp32, steps are 2^-133 (bf16) or 2^-149 whatever the value, and a result may
be flushed to zero. Such a value is off by less than the smallest normal number, TINY:
each P and dS that enters a second product, and each stored result.
"""

import math

import torch

from _step_ref import D, E32, U

TINY = 2.0 ** -126
FEW = 16 * E32     # 2^x, log2, the products by log2(e) and the normalisation: some roundings each


def visible(n, window, sinks, device):
    i = torch.arange(n, device=device)[:, None]
    j = torch.arange(n, device=device)[None, :]
    seen = j <= i
    if window:
        seen &= (i - j < window) | (j < sinks)
    return seen


def heads(QKV, n_q, n_kv):
    """Q [T, n_q, d], K and V [T, n_kv, d] of the fused rows, in 64 bits."""
    G = n_q // n_kv
    x = QKV.to(D).reshape(QKV.shape[0], n_kv, G + 2, -1)
    return x[:, :, :G].reshape(QKV.shape[0], n_q, -1), x[:, :, G], x[:, :, G + 1]


def _sequence_scores(q, k, seen, scale):
    """Scores of [h, n, n] and how far a dot in fp32 may be off, for the visible pairs."""
    s = torch.einsum("qhd,khd->hqk", q, k) * scale
    e = torch.einsum("qhd,khd->hqk", q.abs(), k.abs()) * (abs(scale) * (q.shape[-1] + 4) * E32)
    return s.masked_fill(~seen, -math.inf), e.masked_fill(~seen, 0.0)


def forward(QKV, edges, n_q, n_kv, window, sinks, scale, dtype):
    """O [T, n_q d], lse [n_q, T] and their bounds."""
    T = QKV.shape[0]
    Q, K, V = heads(QKV, n_q, n_kv)
    d = Q.shape[-1]
    O, eO = (torch.zeros(T, n_q, d, dtype=D, device=QKV.device) for _ in range(2))
    lse, el = (torch.zeros(n_q, T, dtype=D, device=QKV.device) for _ in range(2))
    half = U[dtype] if dtype == torch.bfloat16 else 0.0
    for a, b in zip(edges, edges[1:]):
        n = b - a
        if n == 0:
            continue
        G = n_q // n_kv
        k, v = (x[a:b].repeat_interleave(G, 1) for x in (K, V))
        seen = visible(n, window, sinks, QKV.device)
        s, es = _sequence_scores(Q[a:b], k, seen, scale)
        p = s.softmax(-1)
        lse[:, a:b] = s.logsumexp(-1)
        # every term of the sum is off by its exponent's error and some roundings, the sum by its chain
        size = s.masked_fill(~seen, 0.0).abs().amax(-1)
        rel = es.amax(-1) + FEW + 2 * E32 * size + n * E32
        el[:, a:b] = rel + 4 * E32 * lse[:, a:b].abs()
        O[a:b] = torch.einsum("hqk,khd->qhd", p, v)
        weight = torch.einsum("hqk,khd->qhd", p, v.abs())
        err = weight * (half + 2 * rel + n * E32).T[:, :, None]
        err = err + TINY * torch.einsum("hqk,khd->qhd", seen.to(D).expand(n_q, n, n), v.abs())
        eO[a:b] = err + U[dtype] * (O[a:b].abs() + err) + TINY
    return O.reshape(T, -1), lse, eO.reshape(T, -1), el


def backward(dO, QKV, O, lse, edges, n_q, n_kv, window, sinks, scale, dtype):
    """dQKV and its bound, from the O and lse that are given."""
    T = QKV.shape[0]
    Q, K, V = heads(QKV, n_q, n_kv)
    d, G = Q.shape[-1], n_q // n_kv
    dO, O = (x.to(D).reshape(T, n_q, d) for x in (dO, O))
    grad, err = (torch.zeros(T, n_kv, G + 2, d, dtype=D, device=QKV.device) for _ in range(2))
    half = U[dtype] if dtype == torch.bfloat16 else 0.0
    for a, b in zip(edges, edges[1:]):
        n = b - a
        if n == 0:
            continue
        q, g, o, l = Q[a:b], dO[a:b], O[a:b], lse[:, a:b].to(D)[:, :, None]
        k, v = (x[a:b].repeat_interleave(G, 1) for x in (K, V))
        seen = visible(n, window, sinks, QKV.device)
        s, es = _sequence_scores(q, k, seen, scale)
        p = (s - l).exp()
        ep = p * (es + FEW + 2 * E32 * (l.abs() + s.masked_fill(~seen, 0.0).abs())) + TINY * seen
        dot = torch.einsum("qhd,khd->hqk", g, v)
        edot = torch.einsum("qhd,khd->hqk", g.abs(), v.abs()) * ((d + 4) * E32)
        delta = torch.einsum("qhd,qhd->hq", g, o)[:, :, None]
        edelta = torch.einsum("qhd,qhd->hq", g.abs(), o.abs())[:, :, None] * ((d + 4) * E32)
        ds = p * (dot - delta)
        eds = ep * (dot - delta).abs() + (p + ep) * (edot + edelta) + 4 * E32 * ds.abs()
        eds = eds + half * (ds.abs() + eds) + TINY * seen
        epr = ep + half * (p + ep) + TINY * seen
        chain = n * G * E32

        def put(to, out, x, ex, y, f, group):
            """sum over one index of x y, times f, with x's error and the sum's chain; over a group's heads if said"""
            val = torch.einsum(out, x, y) * f
            e = torch.einsum(out, ex + chain * x.abs(), y.abs()) * abs(f)
            val, e = (t.reshape(n, n_kv, G, d) for t in (val, e))
            if group:
                val, e = val.sum(2), e.sum(2)
            e = e + (U[dtype] + 2 * E32) * (val.abs() + e) + TINY
            grad[a:b, :, to], err[a:b, :, to] = val, e

        put(slice(0, G), "hqk,khd->qhd", ds, eds, k, scale, False)
        put(G, "hqk,qhd->khd", ds, eds, q, scale, True)
        put(G + 1, "hqk,qhd->khd", p, epr, g, 1.0, True)
    return grad.reshape(T, -1), err.reshape(T, -1)
