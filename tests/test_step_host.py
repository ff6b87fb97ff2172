"""The training-step operators' refusals and sizes, on the CPU: every call here
is turned down by the library's host checks or the binding's, so none reaches a
kernel (the pointers are never read)."""

import ctypes
import math
import os
import random
import subprocess
import sys

import pytest
import torch

P = ctypes.c_void_p
OK = P(1 << 20)
ODD = P((1 << 20) + 8)
INVALID, SHAPE, ALIGN, WORKSPACE = 1, 2, 3, 4


@pytest.fixture(scope="module")
def L():
    from vocab_ce_gb300 import build
    build.build()
    from vocab_ce_gb300._lib import lib
    return lib()


def test_rmsnorm_forward_refusals(L):
    def call(T=4, h=64, eps=1e-6, dtype=0, X=OK, R=None, w=OK, S=None, Y=OK, Q=None, Qs=None, rstd=OK):
        return L.tp_rmsnorm_forward(X, R, w, T, h, eps, dtype, S, Y, Q, Qs, rstd, None)
    assert call(T=0, X=None, Y=None, rstd=None) == 0
    assert call(T=-1) == SHAPE and call(h=0) == SHAPE and call(h=60) == SHAPE and call(h=16392) == SHAPE
    assert call(dtype=2) == INVALID and call(eps=-1.0) == INVALID and call(eps=float("nan")) == INVALID
    assert call(X=None) == INVALID and call(w=None) == INVALID and call(rstd=None) == INVALID
    assert call(R=OK, S=None) == INVALID          # a sum has to go somewhere
    assert call(Y=None) == INVALID                # neither output
    assert call(Q=OK, Qs=None) == INVALID         # codes without scales
    for name in ("X", "w", "Y", "rstd"):
        assert call(**{name: ODD}) == ALIGN
    assert call(R=ODD, S=OK) == ALIGN and call(Q=ODD, Qs=OK) == ALIGN and call(Q=OK, Qs=ODD) == ALIGN


def test_rmsnorm_backward_refusals(L):
    def call(T=4, h=64, dtype=0, dY=OK, S=OK, w=OK, rstd=OK, dS=None, dX=OK, dw=OK, ws=OK, n=1 << 30):
        return L.tp_rmsnorm_backward(dY, S, w, rstd, dS, T, h, dtype, dX, dw, ws, n, None)
    assert call(T=-1) == SHAPE and call(h=12) == SHAPE and call(dtype=-1) == INVALID
    for name in ("dY", "S", "w", "rstd", "dX"):
        assert call(**{name: None}) == INVALID
        assert call(**{name: ODD}) == ALIGN
    assert call(dS=ODD) == ALIGN and call(dw=ODD) == ALIGN and call(ws=ODD) == ALIGN
    need = L.tpce_rmsnorm_workspace_bytes(4, 64)
    assert need > 0 and call(ws=None) == WORKSPACE and call(n=need - 1) == WORKSPACE
    assert str(need) in L.tpce_last_error().decode()
    assert call(T=0, dY=None, S=None, dX=None, rstd=None, w=None, dw=None, ws=None) == 0


def test_rmsnorm_workspace(L):
    import vocab_ce_gb300 as tp
    assert tp.rmsnorm_workspace_bytes(0, 64) == 0 and tp.rmsnorm_workspace_bytes(-1, 64) == 0
    assert tp.rmsnorm_workspace_bytes(4, 60) == 0
    # one row of fp32 sums for each of a bounded number of blocks
    for T, h in ((1, 8), (7, 1024), (5, 2048), (1 << 20, 16384)):
        n = tp.rmsnorm_workspace_bytes(T, h)
        assert n % (4 * h) == 0 and 1 <= n // (4 * h) <= min(T, 1024)


def test_expert_plan_refusals(L):
    def call(T=4, k=2, E=8, ids=OK, row=OK, source=OK, offsets=OK, ws=None, n=0):
        return L.tp_expert_plan(ids, T, k, E, row, source, offsets, ws, n, None)
    assert call(T=-1) == SHAPE and call(k=0) == SHAPE and call(k=33) == SHAPE
    assert call(E=0) == SHAPE and call(E=1025) == SHAPE and call(T=1 << 30) == SHAPE
    for name in ("ids", "row", "source", "offsets"):
        assert call(**{name: None}) == INVALID
        assert call(**{name: ODD}) == ALIGN
    assert call(T=0, offsets=None) == INVALID
    # few assignments need no workspace; more need E counts for each of at most 256 blocks
    need = L.tpce_expert_plan_workspace_bytes
    assert need(1024, 2, 8) == 0 and need(0, 2, 8) == 0 and need(10_000, 0, 8) == 0
    for T, k, E in ((1025, 2, 8), (16384, 8, 64), (10_000_000, 8, 1024)):
        assert 0 < need(T, k, E) <= 256 * E * 4 and need(T, k, E) % (4 * E) == 0
        assert call(T=T, k=k, E=E) == WORKSPACE and call(T=T, k=k, E=E, ws=OK, n=need(T, k, E) - 1) == WORKSPACE
        assert call(T=T, k=k, E=E, ws=ODD, n=1 << 30) == ALIGN


def test_expert_plan_refuses_overlaps(L):
    # row in the place of ids would make the second pass take ranks for experts
    def call(T, k=2, E=8, ws=None, n=0, **at):
        p = dict(ids=1 << 20, row=2 << 20, source=3 << 20, offsets=4 << 20)
        p.update(at)
        return L.tp_expert_plan(P(p["ids"]), T, k, E, P(p["row"]), P(p["source"]), P(p["offsets"]), ws, n, None)
    for T in (4, 5000):
        bytes_ = 4 * 2 * T
        ws, n = P(5 << 20), L.tpce_expert_plan_workspace_bytes(T, 2, 8)
        for a, b in (("row", "ids"), ("source", "ids"), ("offsets", "ids"), ("source", "row"), ("offsets", "source")):
            base = dict(ids=1 << 20, row=2 << 20, source=3 << 20, offsets=4 << 20)[b]
            for shift in (0, 16, bytes_ - 16):
                assert call(T, ws=ws, n=n, **{a: base + shift}) == INVALID, (a, b, shift)
                assert b"overlap" in L.tpce_last_error()
    for at in (1 << 20, (2 << 20) + 4 * 2 * 5000 - 16, (3 << 20) - 16, 4 << 20):
        assert call(5000, ws=P(at), n=1 << 20) == INVALID and b"overlap" in L.tpce_last_error()
    if not torch.cuda.is_available():      # side by side: what comes next is the launch, which fails without a device
        assert call(4, row=(1 << 20) + 32, source=(1 << 20) + 64, offsets=(1 << 20) + 96) == 5
        assert call(5000, ws=P((4 << 20) + 48), n=1 << 20) == 5


def test_expert_row_refusals(L):
    calls = {
        "dispatch": lambda T=4, h=64, k=2, E=8, dt=0, a=OK, b=OK, c=OK, d=OK:
            L.tp_expert_dispatch_forward(a, b, c, T, h, k, E, dt, d, None),
        "dispatch_backward": lambda T=4, h=64, k=2, E=8, dt=0, a=OK, b=OK, c=OK, d=OK:
            L.tp_expert_dispatch_backward(a, b, T, h, k, dt, d, None),
        "combine": lambda T=4, h=64, k=2, E=8, dt=0, a=OK, b=OK, c=OK, d=OK:
            L.tp_expert_combine_forward(a, b, c, T, h, k, dt, d, None),
        "combine_backward": lambda T=4, h=64, k=2, E=8, dt=0, a=OK, b=OK, c=OK, d=OK, e=OK, f=OK:
            L.tp_expert_combine_backward(a, f, b, c, OK, T, h, k, E, dt, d, e, None),
    }
    for name, call in calls.items():
        assert call(T=0, a=None, d=None) == 0, name
        assert call(T=-1) == SHAPE and call(h=4) == SHAPE and call(h=12) == SHAPE and call(h=(1 << 20) + 8) == SHAPE
        assert call(k=0) == SHAPE and call(k=33) == SHAPE and call(dt=7) == INVALID
        assert call(T=(1 << 31) // 2) == SHAPE
        for p in ("a", "b", "d"):
            assert call(**{p: None}) == INVALID, (name, p)
            assert call(**{p: ODD}) == ALIGN, (name, p)
    for name in ("dispatch", "combine", "combine_backward"):
        assert calls[name](c=None) == INVALID and calls[name](c=ODD) == ALIGN
    for name in ("dispatch", "combine_backward"):
        assert calls[name](E=0) == SHAPE and calls[name](E=1025) == SHAPE
    assert calls["combine_backward"](e=None) == INVALID and calls["combine_backward"](f=ODD) == ALIGN


def test_adamw_refusals(L):
    from vocab_ce_gb300._lib import AdamwTensor

    def call(count=1, lr=1e-3, b1=0.9, b2=0.999, eps=1e-8, step=1, scale=1.0, scalars=None, tensors=True, **kw):
        f = dict(p=1 << 20, master=None, g=1 << 21, m=1 << 22, v=1 << 23, m_scale=1 << 24, v_scale=1 << 25, n=100,
                 weight_decay=0.1, p_dtype=0, g_dtype=0, state_bits=8)
        f.update(kw)
        arr = (AdamwTensor * 1)(AdamwTensor(**f))
        return L.tp_adamw_step(arr if tensors else None, count, lr, b1, b2, eps, step, scale, scalars, None)
    assert call(count=0) == 0 and call(count=0, tensors=False) == 0
    assert call(count=-1) == INVALID and call(tensors=False) == INVALID
    nan, inf = float("nan"), float("inf")
    for bad in (dict(b1=1.0), dict(b1=-0.1), dict(b2=1.0), dict(b2=nan), dict(eps=-1.0), dict(eps=inf), dict(step=0),
                dict(lr=nan), dict(lr=inf), dict(scale=inf), dict(p_dtype=2), dict(g_dtype=5), dict(state_bits=16),
                dict(weight_decay=nan), dict(p=None), dict(g=None), dict(m=None), dict(v=None), dict(m_scale=None),
                dict(v_scale=None), dict(p_dtype=1, master=1 << 26)):
        assert call(**bad) == INVALID, bad
    assert call(n=-1) == SHAPE and call(n=1 << 62) == SHAPE
    for name in ("p", "g", "m", "v", "m_scale", "v_scale", "master"):
        assert call(**{name: (1 << 20) + 4}) == ALIGN, name
    assert call(scalars=P((1 << 20) + 2)) == ALIGN
    # a tensor without values is skipped, whatever its pointers
    assert call(n=0, p=None, g=None, m=None, v=None) == 0


def test_binding_refuses_host_tensors_and_wrong_arguments():
    import vocab_ce_gb300 as tp
    x, w = torch.zeros(4, 64, dtype=torch.bfloat16), torch.ones(64)
    with pytest.raises(ValueError, match="CUDA"):
        tp.tp_rmsnorm_forward(x, w)
    with pytest.raises(ValueError, match="float16"):
        tp.tp_rmsnorm_forward(x.half(), w)
    with pytest.raises(ValueError, match="matrix"):
        tp.tp_rmsnorm_forward(x[0], w)
    with pytest.raises(ValueError, match="CUDA"):
        tp.tp_rmsnorm_backward(x, x, w, torch.ones(4))
    with pytest.raises(ValueError, match="CUDA"):
        tp.tp_expert_plan(torch.zeros(4, 2, dtype=torch.int32), 8)
    plan = {"row": torch.zeros(4, 2, dtype=torch.int32), "offsets": torch.zeros(9, dtype=torch.int32)}
    with pytest.raises(ValueError, match="CUDA"):
        tp.tp_expert_dispatch_forward(x, plan)
    with pytest.raises(ValueError, match="CUDA"):
        tp.adamw_step([x], [x], [tp.adamw_state(x)], lr=1e-3, step=1)
    with pytest.raises(ValueError, match="grads"):
        tp.adamw_step([x], [], [tp.adamw_state(x)], lr=1e-3, step=1)
    with pytest.raises(ValueError, match="fp32 already"):
        tp.adamw_step([w], [w], [tp.adamw_state(w)], lr=1e-3, step=1, masters=[w])
    with pytest.raises(ValueError, match="bits"):
        tp.adamw_state(x, bits=4)


def test_adamw_state_and_scalars():
    import vocab_ce_gb300 as tp
    x = torch.zeros(3, 100, dtype=torch.bfloat16)
    s = tp.adamw_state(x, bits=8)
    assert s["m_q"].dtype == torch.float8_e4m3fn and s["r_q"].shape == x.shape
    assert s["m_scale"].shape == (3,) == s["r_scale"].shape   # 300 values: three groups
    assert tp.adamw_state(x)["v"].dtype == torch.float32
    v = tp.adamw_scalars(1e-3, 10, 0.9, 0.99, grad_scale=0.25)
    want = [1e-3 / (1 - 0.9 ** 10), 1 / math.sqrt(1 - 0.99 ** 10), 1e-3, 0.25]
    assert v.dtype == torch.float32 and torch.equal(v, torch.tensor(want, dtype=torch.float32))
    with pytest.raises(ValueError):
        tp.adamw_scalars(1e-3, 0)


_CALL_WITHOUT_A_DEVICE = """
import ctypes, sys
from vocab_ce_gb300._lib import lib
P = ctypes.c_void_p
p = P(1 << 20)
L = lib()
for h in (64, 256, 264, 512, 8192, 16384):
    for dtype in (0, 1):
        for T in (1, 4, 100_000):
            for r in (None, p):
                assert L.tp_rmsnorm_forward(p, r, p, T, h, 1e-6, dtype, r, p, None, None, p, None) == 5, (h, T)
                assert L.tpce_last_error()
            assert L.tp_rmsnorm_backward(p, p, p, p, None, T, h, dtype, p, None, None, 0, None) == 5, (h, T)
    assert L.tp_expert_combine_forward(p, p, p, 4, h, 2, 0, p, None) == 5
# without tokens an output is set to zero: the text is that failure's, not an earlier one's
assert L.tp_rmsnorm_forward(p, None, p, 4, 60, 1e-6, 0, None, p, None, None, p, None) == 2
assert L.tp_rmsnorm_backward(None, None, None, None, None, 0, 64, 0, None, p, None, 0, None) == 5
assert b"tp_rmsnorm_backward: cuda" in L.tpce_last_error(), L.tpce_last_error()
assert L.tp_expert_plan(None, 0, 2, 8, None, None, p, None, 0, None) == 5
assert b"tp_expert_plan: cuda" in L.tpce_last_error(), L.tpce_last_error()
"""


def test_calls_without_a_device_return_a_status(L):
    # a status code for every layout of the rows: the host arithmetic must not divide by a missing device's SMs
    if torch.cuda.is_available():
        pytest.skip("the pointers are not memory: only where no launch can begin")
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", _CALL_WITHOUT_A_DEVICE], cwd=root, capture_output=True, text=True,
                       timeout=300)
    assert r.returncode == 0, (r.returncode, r.stderr[-2000:])


def _adamw_list(L, *tensors):
    """The status of a step over tensors given as dicts of addresses, as a list or one of many others."""
    from vocab_ce_gb300._lib import AdamwTensor
    return L.tp_adamw_step((AdamwTensor * len(tensors))(*(AdamwTensor(**t) for t in tensors)), len(tensors), 1e-3, 0.9,
                           0.999, 1e-8, 1, 1.0, None, None)


def _adamw_tensor(at, n=300, bits=8, p_dtype=0, g_dtype=0):
    """Every part in a place of its own, 1 MB apart from `at` MB on."""
    names = ["p", "g", "m", "v"] + (["m_scale", "v_scale"] if bits == 8 else []) + (["master"] if p_dtype == 0 else [])
    return dict({k: (at + i) << 20 for i, k in enumerate(names)}, n=n, weight_decay=0.0, p_dtype=p_dtype,
                g_dtype=g_dtype, state_bits=bits)


@pytest.mark.parametrize("others", [0, 3, 30])
def test_adamw_refuses_what_would_be_written_twice(L, others):
    # the others make the list long enough for every way of the check, and stand in no order
    rest = [_adamw_tensor(1000 + 10 * ((7 * i) % others), 1 + 37 * i, (8, 32)[i % 2], i // 2 % 2)
            for i in range(others)]

    def refused(*tensors, says):
        for order in (tensors, tensors[::-1]):
            for at in {0, len(rest) // 2, len(rest)}:
                assert _adamw_list(L, *rest[:at], *order, *rest[at:]) == INVALID, says
                text = L.tpce_last_error().decode()
                assert "overlaps" in text and all(w in text for w in says), (text, says)

    for bits in (8, 32):
        for p_dtype in (0, 1):
            a, b = _adamw_tensor(1, 300, bits, p_dtype), _adamw_tensor(100, 300, bits, p_dtype)
            written = [k for k in a if k in ("p", "m", "v", "m_scale", "v_scale", "master")]
            state, value, grad = (1, 2, 2) if bits == 8 else (4, 2, 2)
            size = {"p": 300 * (2 if p_dtype == 0 else 4), "m": 300 * state, "v": 300 * state, "m_scale": 12,
                    "v_scale": 12, "master": 1200, "g": 600}
            for k in written:
                refused(a, dict(b, **{k: a[k]}), says=[k])                              # the same place
                refused(a, dict(b, p=a[k] + size[k] // 2 // 16 * 16), says=[k, "p"])    # inside it
                refused(a, dict(b, g=a[k]), says=[k, "g"])                              # read while it is written
                refused(dict(a, **{k: a["g"] + 592}), says=[k, "g"])                    # the last values of its own
            refused(dict(a, v=a["m"]), says=["m", "v"])
            refused(a, dict(b, p=a["m"] - 304), says=["p", "m"])                        # from before it into it
            # a large one around small ones
            refused(_adamw_tensor(1, (8 << 20), bits, p_dtype), b, says=["overlaps"])


def test_adamw_accepts_neighbours_and_shared_gradients(L):
    # side by side without a gap, in either order; one gradient for several parameters: what comes next is the launch,
    # which fails where there is no device
    if torch.cuda.is_available():
        pytest.skip("the pointers are not memory: only where no launch can begin")
    for count in (1, 2, 20, 100):
        at, list_ = 1 << 20, []
        for i in range(count):
            n, t = 16 * (1 + i % 9), dict(weight_decay=0.0, p_dtype=0, g_dtype=0, state_bits=8, n=16 * (1 + i % 9))
            for k, size in (("p", 2 * n), ("master", 4 * n), ("m", n), ("v", n), ("m_scale", 16), ("v_scale", 16)):
                t[k] = at
                at += size
            list_.append(t)
        for t in list_:
            t["g"] = at
        for order in (list_, list_[::-1], list_[::2] + list_[1::2]):
            assert _adamw_list(L, *order) == 5, L.tpce_last_error()


def test_adamw_overlaps_of_random_lists(L):
    # against every pair compared
    if torch.cuda.is_available():
        pytest.skip("the pointers are not memory: only where no launch can begin")
    rng = random.Random(0)
    seen = [0, 0]
    for _ in range(400):
        count, room = rng.choice([1, 2, 5, 12, 40]), rng.choice([20, 2000, 40_000])
        list_, ranges = [], []
        for i in range(count):
            n, bits = rng.randint(0, 400), rng.choice([8, 32])
            t = dict(n=n, weight_decay=0.0, p_dtype=rng.randint(0, 1), g_dtype=rng.randint(0, 1), state_bits=bits)
            state, scales = (1, 4 * -(-n // 128)) if bits == 8 else (4, 0)
            sizes = {"p": n * (2, 4)[t["p_dtype"]], "m": n * state, "v": n * state, "g": n * (2, 4)[t["g_dtype"]],
                     "m_scale": scales, "v_scale": scales}
            if t["p_dtype"] == 0 and rng.random() < 0.5:
                sizes["master"] = 4 * n
            for k, size in sizes.items():
                t[k] = (1 << 24) + 16 * rng.randrange(room) + 16 * room * i * (rng.random() < 0.7)
                if size:
                    ranges.append((t[k], t[k] + size, k == "g"))
            list_.append(t)
        bad = any(a[0] < b[1] and b[0] < a[1] and not (a[2] and b[2])
                  for i, a in enumerate(ranges) for b in ranges[:i])
        want = INVALID if bad else 5 if ranges else 0
        assert _adamw_list(L, *list_) == want, L.tpce_last_error()
        seen[bad] += 1
    assert min(seen) > 40, seen


def test_adamw_rounding_is_nearest_or_random(L):
    import vocab_ce_gb300 as tp
    for bits in (32 | 256, 16 | 256, 256, 8 | 512):
        assert _adamw_list(L, dict(_adamw_tensor(1), state_bits=bits)) == INVALID, bits
    t = dict(_adamw_tensor(1), state_bits=8 | 256)
    assert _adamw_list(L, t, dict(_adamw_tensor(20), v=t["v"])) == INVALID and b"overlaps" in L.tpce_last_error()
    assert _adamw_list(L, dict(t, m_scale=None)) == INVALID
    with pytest.raises(ValueError, match="rounding"):
        tp.adamw_step([], [], [], lr=1e-3, step=1, rounding="up")
