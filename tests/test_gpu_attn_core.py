"""The attention core and its gradients against 64-bit forms within derived bounds
(_attn_ref): one token to several tiles, lengths around a tile's edge, packed
sequences with empty ones and rows of none, windows of one key to more than there
are, first keys that stay visible, heads that share keys or do not, head widths
from 8 to 128; infinities and NaN where a query does not see them; offsets that
fall; rows past 32 bits; another stream, a graph, equal bits each time.
"""

import math

import pytest
import torch

import _attn_ref as ref
import vocab_ce_gb300 as tp
from _parity import gpu_or_skip
from _step_ref import D, near

pytestmark = pytest.mark.gpu
TYPES = [torch.bfloat16, torch.float32]
BF, F32 = TYPES
# (lengths, rows before, rows behind, n_kv, group, d, window, sinks)
CASES = [
    ((1,), 0, 0, 1, 1, 8, 0, 0), ((1,), 3, 2, 2, 2, 128, 1, 0), ((2, 1, 0, 3), 0, 0, 1, 2, 64, 0, 0),
    ((17,), 0, 0, 8, 8, 128, 0, 0), ((63, 64, 65), 0, 5, 1, 3, 16, 0, 0), ((127, 128, 129), 1, 0, 2, 1, 40, 0, 0),
    ((300,), 0, 0, 1, 8, 128, 0, 0), ((255, 0, 257), 0, 140, 2, 2, 72, 0, 0), ((700,), 0, 0, 1, 1, 96, 0, 0),
    ((200,), 0, 0, 2, 1, 64, 1, 0), ((200,), 0, 0, 1, 2, 64, 1, 1), ((330, 40), 7, 0, 1, 3, 80, 5, 4),
    ((400,), 0, 0, 1, 2, 128, 64, 0), ((513,), 0, 3, 1, 1, 128, 128, 64), ((600, 130), 0, 0, 1, 2, 96, 100, 130),
    ((385,), 0, 0, 1, 4, 128, 127, 1), ((641,), 0, 0, 1, 1, 64, 129, 200), ((150,), 0, 0, 1, 2, 24, 150, 3),
    ((150,), 0, 0, 1, 2, 32, 10 ** 12, 3), ((260,), 0, 0, 1, 2, 112, 9, 10 ** 12), ((1024,), 0, 0, 1, 1, 128, 0, 0),
    ((5,) * 70, 0, 0, 1, 2, 64, 0, 0), ((130,) * 9 + (1,), 2, 2, 2, 3, 128, 50, 2),
]


def make(lengths, before, behind, n_kv, G, d, dtype, seed, std=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    edges = [before]
    for n in lengths:
        edges.append(edges[-1] + n)
    T, n_q = edges[-1] + behind, n_kv * G
    QKV = (std * torch.randn(T, (n_q + 2 * n_kv) * d, generator=g, device="cuda")).to(dtype)
    dO = torch.randn(T, n_q * d, generator=g, device="cuda").to(dtype)
    return QKV, dO, edges, torch.tensor(edges, dtype=torch.int32, device="cuda")


def bits(x):
    return x.contiguous().view(torch.uint8)


def check(QKV, dO, edges, offsets, n_q, n_kv, window, sinks, dtype, scale=None):
    d = QKV.shape[1] // (n_q + 2 * n_kv)
    f = 1.0 / math.sqrt(d) if scale is None else scale
    kw = dict(offsets=offsets, window=window, sinks=sinks, scale=scale)
    O, lse, eO, el = ref.forward(QKV, edges, n_q, n_kv, window, sinks, f, dtype)
    got = tp.tp_attn_core_forward(QKV, n_q, n_kv, **kw)
    near(got["lse"], lse, el, "lse")
    near(got["O"], O, eO, "O")
    again = tp.tp_attn_core_forward(QKV, n_q, n_kv, **kw)
    assert torch.equal(got["O"], again["O"]) and torch.equal(got["lse"], again["lse"])
    given = O.to(dtype), lse.float()
    want, err = ref.backward(dO, QKV, *given, edges, n_q, n_kv, window, sinks, f, dtype)
    grad = tp.tp_attn_core_backward(dO, QKV, *given, n_q, n_kv, **kw)
    G = n_q // n_kv
    for name, at in (("dQ", slice(0, G)), ("dK", G), ("dV", G + 1)):
        x, w, e = (t.reshape(-1, n_kv, G + 2, d)[:, :, at] for t in (grad, want, err))
        near(x, w, e, name)
    again = tp.tp_attn_core_backward(dO, QKV, *given, n_q, n_kv, **kw)
    assert torch.equal(grad, again)
    inside = torch.zeros(len(QKV), dtype=torch.bool, device="cuda")
    inside[edges[0]:edges[-1]] = True
    for x in (got["O"], got["lse"].T, grad):
        assert not bits(x[~inside]).any()
    assert tp.device_status() == 0


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("lengths,before,behind,n_kv,G,d,window,sinks", CASES)
def test_forward_and_gradients(lengths, before, behind, n_kv, G, d, window, sinks, dtype):
    gpu_or_skip()
    QKV, dO, edges, offsets = make(lengths, before, behind, n_kv, G, d, dtype, sum(lengths) + d)
    check(QKV, dO, edges, offsets, n_kv * G, n_kv, min(window, 10 ** 9), sinks, dtype)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("T", [1, 64, 130, 500])
def test_one_sequence_without_offsets(T, dtype):
    gpu_or_skip()
    QKV, dO, edges, _ = make((T,), 0, 0, 2, 2, 64, dtype, T)
    check(QKV, dO, edges, None, 4, 2, 0, 0, dtype)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("scale,std", [(0.0, 1.0), (-0.3, 1.0), (1.0, 3.0), (4.0, 4.0)])
def test_scales(scale, std, dtype):
    # large scores: a row's maximum moves far from tile to tile, and most of P vanishes
    gpu_or_skip()
    QKV, dO, edges, offsets = make((400, 77), 0, 0, 1, 2, 64, dtype, 5, std)
    check(QKV, dO, edges, offsets, 2, 1, 0, 0, dtype, scale)


def test_rising_scores():
    # every tile's maximum is above the one before, by a little and by much
    gpu_or_skip()
    for step in (0.05, 0.5, 5.0):
        QKV, dO, edges, offsets = make((640,), 0, 0, 1, 1, 64, BF, 6, 0.1)
        ramp = torch.arange(640, device="cuda") * (step / 128)
        QKV[:, 0], QKV[:, 64] = 8.0, ramp.to(BF)
        check(QKV, dO, edges, offsets, 1, 1, 0, 0, BF)


def put_bad(x, rows, value):
    x[rows] = value
    return x


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("value", [math.nan, math.inf, -math.inf])
def test_what_is_not_seen_does_not_reach(value, dtype):
    gpu_or_skip()
    n_q, n_kv, d, at, window = 2, 1, 64, 150, 40
    for w, sinks, hidden in ((0, 0, lambda i: i < at), (window, 0, lambda i: (i < at) | (i >= at + window))):
        QKV, dO, edges, offsets = make((333, 70), 0, 9, n_kv, 2, d, dtype, 7)
        i = torch.arange(333, device="cuda")
        free = torch.cat([hidden(i), torch.ones(70, dtype=torch.bool, device="cuda"),
                          torch.zeros(9, dtype=torch.bool, device="cuda")])
        kw = dict(offsets=offsets, window=w, sinks=sinks)
        good = tp.tp_attn_core_forward(QKV, n_q, n_kv, **kw)
        gO, glse, _, _ = ref.forward(QKV, edges, n_q, n_kv, w, sinks, d ** -0.5, dtype)
        want = tp.tp_attn_core_backward(dO, QKV, gO.to(dtype), glse.float(), n_q, n_kv, **kw)
        eO = ref.forward(QKV, edges, n_q, n_kv, w, sinks, d ** -0.5, dtype)[2]
        ew = ref.backward(dO, QKV, gO.to(dtype), glse.float(), edges, n_q, n_kv, w, sinks, d ** -0.5, dtype)
        # a key and its value, and rows behind the last sequence
        bad = QKV.clone()
        bad[at, n_q * d:] = value
        bad[403:] = math.nan
        got = tp.tp_attn_core_forward(bad, n_q, n_kv, **kw)
        near(got["O"][free], gO[free], eO[free], "O")
        near(got["lse"][:, free], good["lse"][:, free], 2.0 ** -18, "lse")
        seen = ~free
        seen[333:] = False
        assert not torch.isfinite(got["O"][seen].float()).any(1).any() or not math.isnan(value)
        assert not bits(got["O"][403:]).any()
        # the same in the backward: queries that do not see the key
        badO, dbad = dO.clone(), None
        badO[403:] = math.nan
        bad_lse, bad_out = glse.float(), gO.to(dtype)
        dbad = tp.tp_attn_core_backward(badO, bad, bad_out, bad_lse, n_q, n_kv, **kw)
        q = slice(0, n_q * d)
        near(dbad[free][:, q], ew[0][free][:, q], ew[1][free][:, q], "dQ")
        assert torch.isfinite(want).all() and not bits(dbad[403:]).any()
        # a query, and its upstream gradient: keys that it does not see
        bad = QKV.clone()
        bad[at, :n_q * d] = value
        badO[at] = value
        dbad = tp.tp_attn_core_backward(badO, bad, bad_out, bad_lse, n_q, n_kv, **kw)
        apart = (i > at) | ((i <= at - w) if w else False)
        apart = torch.cat([apart, torch.ones(70, dtype=torch.bool, device="cuda"),
                           torch.zeros(9, dtype=torch.bool, device="cuda")])
        kv = slice(n_q * d, None)
        near(dbad[apart][:, kv], ew[0][apart][:, kv], ew[1][apart][:, kv], "dK, dV")
        other = torch.arange(len(QKV), device="cuda") != at
        other[403:] = False
        near(dbad[other][:, q], ew[0][other][:, q], ew[1][other][:, q], "dQ of other queries")


def test_gradients_against_differences():
    gpu_or_skip()
    n_q, n_kv, d, w, sinks = 4, 2, 16, 20, 3
    QKV, dO, edges, offsets = make((70, 30), 0, 0, n_kv, 2, d, F32, 8)
    kw = dict(offsets=offsets, window=w, sinks=sinks)
    f = tp.tp_attn_core_forward(QKV, n_q, n_kv, **kw)
    grad = tp.tp_attn_core_backward(dO, QKV, f["O"], f["lse"], n_q, n_kv, **kw)

    def loss(x):
        return (tp.tp_attn_core_forward(x, n_q, n_kv, **kw)["O"].to(D) * dO.to(D)).sum()

    eO = ref.forward(QKV, edges, n_q, n_kv, w, sinks, d ** -0.5, F32)[2]
    noise = (eO * dO.to(D).abs()).sum().item()
    for r, c in [(0, 3), (25, 20), (69, 40), (2, 66), (40, 100), (99, 70), (70, 127), (3, 90)]:
        step = 2.0 ** -6
        hi, mid, lo = QKV.clone(), QKV.clone(), QKV.clone()
        hi[r, c] += step
        lo[r, c] -= step
        hi2, lo2 = QKV.clone(), QKV.clone()
        hi2[r, c] += 2 * step
        lo2[r, c] -= 2 * step
        a, b = (loss(hi) - loss(lo)).item() / (2 * step), (loss(hi2) - loss(lo2)).item() / (4 * step)
        # the difference's error is a third of what a twice as long one is off by, once more for higher terms
        slack = 2 * abs(b - a) / 3 + 2 * noise / step
        assert abs((4 * a - b) / 3 - grad[r, c].item()) <= slack + 1e-6, (r, c)


def test_offsets_that_fall_or_lie_outside():
    gpu_or_skip()
    QKV, dO, _, _ = make((200,), 0, 0, 1, 2, 64, BF, 9)
    assert tp.device_status() == 0
    for bad, good in (([0, 100, 50, 200], [0, 100, 100, 200]), ([-5, 80, 10 ** 6], [0, 80, 200]),
                      ([300, 400], [200, 200]), ([0, -7, 30], [0, 0, 30])):
        kw = [dict(offsets=torch.tensor(x, dtype=torch.int32, device="cuda")) for x in (bad, good)]
        a = tp.tp_attn_core_forward(QKV, 2, 1, **kw[0])
        assert tp.device_status() == 1
        b = tp.tp_attn_core_forward(QKV, 2, 1, **kw[1])
        ga = tp.tp_attn_core_backward(dO, QKV, b["O"], b["lse"], 2, 1, **kw[0])
        assert tp.device_status() == 1
        gb = tp.tp_attn_core_backward(dO, QKV, b["O"], b["lse"], 2, 1, **kw[1])
        assert torch.equal(a["O"], b["O"]) and torch.equal(a["lse"], b["lse"]) and torch.equal(ga, gb)
        assert tp.device_status() == 0


def test_rows_past_32_bits():
    gpu_or_skip()
    n_q, n_kv, d, w = 16, 16, 64, 33
    ld = (n_q + 2 * n_kv) * d
    T = (1 << 31) // ld + 400
    QKV = torch.zeros(T, ld, dtype=BF, device="cuda")
    few = 260
    tail, dtail, _, _ = make((few,), 0, 0, n_kv, 1, d, BF, 10)
    QKV[T - few:] = tail
    edges = [0, 3, T - few, T]
    offsets = torch.tensor(edges, dtype=torch.int32, device="cuda")
    got = tp.tp_attn_core_forward(QKV, n_q, n_kv, offsets=offsets, window=w)
    want = tp.tp_attn_core_forward(tail, n_q, n_kv, window=w)
    assert torch.equal(got["O"][T - few:], want["O"]) and torch.equal(got["lse"][:, T - few:], want["lse"])
    assert not got["O"][:T - few].any()
    dO = torch.zeros(T, n_q * d, dtype=BF, device="cuda")
    dO[T - few:] = dtail
    grad = tp.tp_attn_core_backward(dO, QKV, got["O"], got["lse"], n_q, n_kv, offsets=offsets, window=w)
    small = tp.tp_attn_core_backward(dtail, tail, want["O"], want["lse"], n_q, n_kv, window=w)
    assert torch.equal(grad[T - few:], small)
    assert not any(bool(grad[i:i + 100_000].any()) for i in range(0, T - few, 100_000) if i + 100_000 <= T - few)


def test_another_stream_and_given_outputs():
    gpu_or_skip()
    QKV, dO, _, offsets = make((300, 45), 0, 0, 2, 4, 128, BF, 11)
    kw = dict(offsets=offsets, window=90, sinks=4)
    f = tp.tp_attn_core_forward(QKV, 8, 2, **kw)
    g = tp.tp_attn_core_backward(dO, QKV, f["O"], f["lse"], 8, 2, **kw)
    out = {k: torch.full_like(v, math.nan) for k, v in f.items()}
    dQKV = torch.full_like(QKV, math.nan)
    ws = torch.full((tp.attn_core_workspace_bytes(345, 8),), 0xff, dtype=torch.uint8, device="cuda")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    r = tp.tp_attn_core_forward(QKV, 8, 2, out=out, stream=s, **kw)
    tp.tp_attn_core_backward(dO, QKV, r["O"], r["lse"], 8, 2, out=dQKV, ws=ws, stream=s, **kw)
    s.synchronize()
    assert r["O"] is out["O"] and r["lse"] is out["lse"]
    assert torch.equal(out["O"], f["O"]) and torch.equal(out["lse"], f["lse"]) and torch.equal(dQKV, g)
    assert (out["O"]._version, out["lse"]._version, QKV._version, dO._version) == (1, 1, 0, 0)


def test_in_a_graph_with_other_lengths():
    gpu_or_skip()
    QKV, dO, _, offsets = make((100, 100, 100), 0, 0, 1, 2, 64, BF, 12)
    out = tp.tp_attn_core_forward(QKV, 2, 1, offsets=offsets, window=70, sinks=2)
    dQKV = torch.empty_like(QKV)
    ws = torch.empty(tp.attn_core_workspace_bytes(300, 2), dtype=torch.uint8, device="cuda")

    def step():
        tp.tp_attn_core_forward(QKV, 2, 1, offsets=offsets, window=70, sinks=2, out=out)
        tp.tp_attn_core_backward(dO, QKV, out["O"], out["lse"], 2, 1, offsets=offsets, window=70, sinks=2, out=dQKV,
                                 ws=ws)

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
    torch.cuda.current_stream().wait_stream(s)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for seed, edges in ((13, [0, 1, 299, 300]), (14, [10, 10, 200, 250])):
        x, y, _, _ = make((300,), 0, 0, 1, 2, 64, BF, seed)
        QKV.copy_(x)
        dO.copy_(y)
        offsets.copy_(torch.tensor(edges, dtype=torch.int32))
        g.replay()
        torch.cuda.synchronize()
        f = tp.tp_attn_core_forward(QKV, 2, 1, offsets=offsets, window=70, sinks=2)
        assert torch.equal(out["O"], f["O"]) and torch.equal(out["lse"], f["lse"])
        assert torch.equal(dQKV, tp.tp_attn_core_backward(dO, QKV, f["O"], f["lse"], 2, 1, offsets=offsets, window=70,
                                                          sinks=2))


def test_no_tokens():
    gpu_or_skip()
    QKV = torch.empty(0, 4 * 64, dtype=BF, device="cuda")
    f = tp.tp_attn_core_forward(QKV, 2, 1)
    assert f["O"].shape == (0, 128) and f["lse"].shape == (2, 0)
    assert tp.tp_attn_core_backward(f["O"], QKV, f["O"], f["lse"], 2, 1).shape == QKV.shape


def test_tensors_that_are_refused():
    gpu_or_skip()
    QKV, dO, _, offsets = make((20,), 0, 0, 1, 2, 64, BF, 15)
    f = tp.tp_attn_core_forward(QKV, 2, 1)
    for bad in (QKV.half(), QKV.cpu(), QKV[:, :192], QKV[0], QKV.T):
        with pytest.raises(ValueError):
            tp.tp_attn_core_forward(bad, 2, 1, out={"O": f["O"]})
    for heads in ((0, 1), (2, 0), (3, 2), (-2, 1)):
        with pytest.raises(ValueError):
            tp.tp_attn_core_forward(QKV, *heads)
    for bad in (offsets.long(), offsets.cpu(), offsets[:1], offsets.reshape(1, 2)):
        with pytest.raises(ValueError):
            tp.tp_attn_core_forward(QKV, 2, 1, offsets=bad)
    for kw in ({"window": -1}, {"sinks": -1}, {"scale": math.inf}, {"scale": math.nan}):
        with pytest.raises(tp.TpceError):
            tp.tp_attn_core_forward(QKV, 2, 1, **kw)
    with pytest.raises(tp.TpceError, match="head width"):
        tp.tp_attn_core_forward(torch.zeros(4, 4 * 136, dtype=BF, device="cuda"), 2, 1)
    with pytest.raises(tp.TpceError, match="head width"):
        tp.tp_attn_core_forward(torch.zeros(4, 4 * 12, dtype=BF, device="cuda"), 2, 1)
    for i, bad in ((0, dO.float()), (0, dO[:10]), (2, f["O"].float()), (3, f["lse"].T), (3, f["lse"].bfloat16())):
        args = [dO, QKV, f["O"], f["lse"]]
        args[i] = bad
        with pytest.raises(ValueError):
            tp.tp_attn_core_backward(*args, 2, 1)
    with pytest.raises(ValueError):
        tp.tp_attn_core_backward(dO, QKV, f["O"], f["lse"], 2, 1, out=dO)
    with pytest.raises(tp.TpceError, match="overlap"):
        tp.tp_attn_core_backward(dO, QKV, f["O"], f["lse"], 2, 1, out=QKV)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("lengths,n_kv,G,d,window,sinks", [
    ((70,), 1, 1, 64, 0, 0),        # two steps on two blocks
    ((130,), 1, 1, 8, 0, 0),        # three on four: one has none
    ((500,), 1, 1, 128, 0, 0),      # eight on eight
    ((600, 3), 1, 2, 40, 0, 0),
    ((1, 64, 65, 300), 1, 1, 96, 0, 0),
    ((1000,), 2, 2, 64, 0, 0),      # four, of more blocks than run at once
    ((700,), 1, 3, 64, 100, 5),
])
def test_tiles_that_blocks_share(lengths, n_kv, G, d, window, sinks, dtype):
    # fp32, and bf16 with a scale that is not positive: calls with few tiles for the SMs
    gpu_or_skip()
    QKV, dO, edges, offsets = make(lengths, 0, 2, n_kv, G, d, dtype, 11)
    check(QKV, dO, edges, offsets, n_kv * G, n_kv, window, sinks, dtype, 0.2 if dtype == F32 else -0.2)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("n_kv,G,d,window,sinks", [(1, 2, 64, 0, 0), (2, 1, 8, 3, 1)])
def test_many_sequences(n_kv, G, d, window, sinks, dtype):
    # more than a lane, and than a warp, looks at in a step; blocks that take many tiles; rows before and behind
    gpu_or_skip()
    lengths = tuple((7 * i * i + 3 * i) % 23 if i % 5 else 0 for i in range(601)) + (200,) + (1,) * 300
    QKV, dO, edges, offsets = make(lengths, 3, 4, n_kv, G, d, dtype, 12)
    check(QKV, dO, edges, offsets, n_kv * G, n_kv, window, sinks, dtype)


@pytest.mark.parametrize("dtype", TYPES)
def test_offsets_that_fall_among_many(dtype):
    gpu_or_skip()
    lengths = (5, 0, 3) * 100
    QKV, dO, edges, offsets = make(lengths, 0, 0, 1, 1, 16, dtype, 13)
    good = tp.tp_attn_core_forward(QKV, 1, 1, offsets=offsets)
    bad = offsets.clone()
    at = 140  # an empty sequence's end: read as the one before, the same sequences
    assert edges[at - 1] == edges[at]
    bad[at] = -5
    got = tp.tp_attn_core_forward(QKV, 1, 1, offsets=bad)
    assert tp.device_status() != 0 and tp.device_status() == 0
    assert torch.equal(got["O"], good["O"]) and torch.equal(got["lse"], good["lse"])


def test_the_most_sequences():
    # nearly all of them empty: passing them takes part of the time that the kernel's other warps wait
    gpu_or_skip()
    n, T = 1 << 26, 100
    QKV, dO, _, _ = make((T,), 0, 0, 1, 1, 64, BF, 14)
    offsets = torch.zeros(n + 1, dtype=torch.int32, device="cuda")
    offsets[n // 2 + 1:], offsets[-1] = 70, T
    few = torch.tensor([0, 70, T], dtype=torch.int32, device="cuda")
    got, want = (tp.tp_attn_core_forward(QKV, 1, 1, offsets=x) for x in (offsets, few))
    assert torch.equal(got["O"], want["O"]) and torch.equal(got["lse"], want["lse"])
    a, b = (tp.tp_attn_core_backward(dO, QKV, want["O"], want["lse"], 1, 1, offsets=x) for x in (offsets, few))
    assert torch.equal(a, b) and tp.device_status() == 0


def test_offsets_that_are_part_of_a_vector():
    gpu_or_skip()
    QKV, dO, edges, _ = make((90, 30, 50), 0, 0, 1, 2, 64, BF, 15)
    longer = torch.tensor([7] + edges + [9], dtype=torch.int32, device="cuda")
    part, whole = longer[1:-1], torch.tensor(edges, dtype=torch.int32, device="cuda")
    assert part.data_ptr() % 16
    f, w = (tp.tp_attn_core_forward(QKV, 2, 1, offsets=x) for x in (part, whole))
    assert torch.equal(f["O"], w["O"]) and torch.equal(f["lse"], w["lse"])
    a, b = (tp.tp_attn_core_backward(dO, QKV, w["O"], w["lse"], 2, 1, offsets=x) for x in (part, whole))
    assert torch.equal(a, b) and tp.device_status() == 0
