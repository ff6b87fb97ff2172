"""Plain 64-bit forms of the training-step operators, and what the tests allow.

A stored result is rounded once, by at most half a step: U[dtype] relative to
its value. Sums are taken in fp32; a sum of positive or mixed terms whose
longest chain of additions is c is off by at most c 2^-24 times the sum of the
terms' absolute values (each addition by half a step of the partial sum). An
e4m3 code is off by 2^-4 of its value, or by half the smallest step, 2^-10, in
units of the scale.
"""

import torch

D = torch.float64
U = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}
E32 = 2.0 ** -24
E4M3_HALF, E4M3_TINY = 2.0 ** -4, 2.0 ** -10
GROUP = 128
MIN_SCALE = 2.0 ** -126


def groups(x):
    """The last dimension as groups of 128, the last one filled with zeros."""
    x = torch.nn.functional.pad(x, (0, -x.shape[-1] % GROUP))
    return x.reshape(*x.shape[:-1], -1, GROUP)


def spread(scale, n):
    """Each value's scale."""
    return scale.to(D).repeat_interleave(GROUP, -1)[..., :n]


def group_scale(x):
    """The scale that a group of x should have (x: any float type, last dimension grouped)."""
    a = groups(x.to(D)).abs()
    a = torch.where(torch.isfinite(a), a, 0.0)
    return (a.amax(-1) / 448.0).clamp_min(MIN_SCALE)


def near(got, want, tol, what):
    got, want = got.to(D), want.to(D)
    assert got.shape == want.shape, (what, got.shape, want.shape)
    if not got.numel():
        return
    bad = ~((got - want).abs() <= tol)
    if bad.any():
        at = torch.nonzero(bad)[0].tolist()
        i = tuple(at)
        t = tol if not torch.is_tensor(tol) else tol.expand(got.shape)[i].item()
        raise AssertionError(f"{what}: {int(bad.sum())} values off; first at {at}: {got[i].item()} for "
                             f"{want[i].item()}, allowed {t}")


def codes_near(q, scale, want, err, what):
    """Codes and scales of `want`, itself known up to `err`."""
    n = want.shape[-1]
    top = groups(err.expand(want.shape)).amax(-1)
    near(scale, group_scale(want), top / 448.0 + 2 * E32 * scale.to(D) + 2.0 ** -149, what + " scale")
    s = spread(scale, n)
    # the value's own error, the rounding of value / scale, and the code's half step
    near(q.float().to(D) * s, want, err + (E4M3_HALF + 4 * E32) * (want.abs() + err) + E4M3_TINY * s, what)


# ------------------------------------------------------------------ norm
def norm_forward(S, w, eps):
    x = S.to(D)
    rstd = (x.pow(2).mean(-1) + eps).pow(-0.5)
    return x * rstd[:, None] * w.to(D), rstd


def norm_backward(dY, S, w, eps, dS=None):
    x, dy = S.to(D), dY.to(D)
    rstd = (x.pow(2).mean(-1, keepdim=True) + eps).pow(-0.5)
    xh, g = x * rstd, dy * w.to(D)
    dX = rstd * (g - xh * (g * xh).mean(-1, keepdim=True))
    return (dX if dS is None else dX + dS.to(D)), (dy * xh).sum(0)


# ------------------------------------------------------------------ experts
def plan(ids, E):
    """row, source, offsets of the stable sort, one assignment after the other."""
    T, k = ids.shape
    by = [[] for _ in range(E)]
    for i, e in enumerate(ids.reshape(-1).tolist()):
        if 0 <= e < E:
            by[e].append(i)
    row, source, offsets = [-1] * (T * k), [], [0]
    for one in by:
        for i in one:
            row[i] = len(source)
            source.append(i)
        offsets.append(len(source))
    source += [-1] * (T * k - len(source))
    return {"row": torch.tensor(row, dtype=torch.int32).reshape(T, k),
            "source": torch.tensor(source, dtype=torch.int32), "offsets": torch.tensor(offsets, dtype=torch.int32)}


# ------------------------------------------------------------------ AdamW
def adamw(p, g, m, v, lr, step, b1, b2, eps, wd, grad_scale):
    """All arguments in 64 bits; returns p, m, v and the size of the terms that p's update adds."""
    g = g * grad_scale
    m = b1 * m + (1 - b1) * g
    v = b2 * v + (1 - b2) * g * g
    u = lr * (m / (1 - b1 ** step)) / ((v / (1 - b2 ** step)).sqrt() + eps)
    return p - lr * wd * p - u, m, v, u.abs()
