"""The attention core in bf16 where a block takes several pairs of tiles or units of
work: more of them than there are SMs, against the 64-bit forms and their bounds
(_attn_ref); and where several of a block's have results that are not finite, which
it computes again: what is masked must not reach there either.
Windows past 32 bits, the longest sequence, and calls on several streams at once.
"""

import math

import pytest
import torch

import _attn_ref as ref
import vocab_ce_gb300 as tp
from _parity import gpu_or_skip
from _step_ref import near
from test_gpu_attn_core import BF, F32, check, make

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("lengths,behind,n_kv,G,d,window,sinks", [
    ((3000,), 0, 4, 4, 128, 0, 0),              # 192 pairs of heads, 480 units
    ((1700, 1250, 50), 9, 6, 3, 96, 0, 0),      # pairs of neighbouring tiles
    ((3000,), 0, 4, 4, 64, 500, 4),
    ((2100, 1, 899), 3, 12, 1, 128, 129, 200),
    ((300,) * 40, 0, 2, 4, 128, 0, 0),          # 480 pairs
])
def test_several_units_a_block(lengths, behind, n_kv, G, d, window, sinks):
    gpu_or_skip()
    QKV, dO, edges, offsets = make(lengths, 0, behind, n_kv, G, d, BF, 41)
    check(QKV, dO, edges, offsets, n_kv * G, n_kv, window, sinks, BF)


@pytest.mark.parametrize("value", [math.nan, math.inf])
@pytest.mark.parametrize("n_kv,G,window,bad", [
    (4, 4, 300, (600, 2000)), (4, 4, 0, (2000,)), (6, 3, 300, (700, 701, 2900)),
])
def test_what_is_not_seen_does_not_reach_in_several_units(n_kv, G, window, bad, value):
    gpu_or_skip()
    T, d, n_q = 3000, 128, n_kv * G
    QKV, dO, edges, _ = make((T,), 0, 0, n_kv, G, d, BF, 42)
    kw = dict(window=window)
    O, lse, eO, el = ref.forward(QKV, edges, n_q, n_kv, window, 0, d ** -0.5, BF)
    given = O.to(BF), lse.float()
    want, err = ref.backward(dO, QKV, *given, edges, n_q, n_kv, window, 0, d ** -0.5, BF)
    i = torch.arange(T, device="cuda")
    reach = window or T
    heads = torch.arange(QKV.shape[1], device="cuda") // d % (G + 2)
    # keys and values that only some queries see
    x = QKV.clone()
    for p in bad:
        x[p, heads >= G] = value
    sees = torch.zeros(T, dtype=torch.bool, device="cuda")
    for p in bad:
        sees |= (i >= p) & (i < p + reach)
    got = tp.tp_attn_core_forward(x, n_q, n_kv, **kw)
    near(got["O"][~sees], O[~sees], eO[~sees], "O")
    near(got["lse"][:, ~sees], lse[:, ~sees], el[:, ~sees], "lse")
    if math.isnan(value):
        assert got["O"][sees].isnan().all() and got["lse"][:, sees].isnan().all()
    again = tp.tp_attn_core_forward(x, n_q, n_kv, **kw)
    assert torch.equal(got["O"].view(torch.int16), again["O"].view(torch.int16))
    grad = tp.tp_attn_core_backward(dO, x, *given, n_q, n_kv, **kw)
    q, kv = heads < G, heads >= G
    near(grad[~sees][:, q], want[~sees][:, q], err[~sees][:, q], "dQ")
    # keys whose queries all see nothing of it
    far = torch.ones(T, dtype=torch.bool, device="cuda")
    for p in bad:
        far &= (i <= p - reach) | (i >= p + reach)
    near(grad[far][:, kv], want[far][:, kv], err[far][:, kv], "dK, dV")
    again = tp.tp_attn_core_backward(dO, x, *given, n_q, n_kv, **kw)
    assert torch.equal(grad.view(torch.int16), again.view(torch.int16))
    # queries, and what comes back to them
    x, g = QKV.clone(), dO.clone()
    apart = torch.ones(T, dtype=torch.bool, device="cuda")
    other = torch.ones(T, dtype=torch.bool, device="cuda")
    for p in bad:
        x[p, heads < G] = value
        g[p] = value
        apart &= (i > p) | (i <= p - reach)
        other &= i != p
    grad = tp.tp_attn_core_backward(g, x, *given, n_q, n_kv, **kw)
    near(grad[apart][:, kv], want[apart][:, kv], err[apart][:, kv], "dK, dV of others")
    near(grad[other][:, q], want[other][:, q], err[other][:, q], "dQ of others")
    assert tp.device_status() == 0


def test_more_pairs_a_block_than_it_has_bits_for():
    # 512 rounds of pairs have a bit each that says that a tile is computed again; the next ones share them
    gpu_or_skip()
    n, d = 100_000, 64
    QKV, _, _, _ = make((2 * n,), 0, 0, 1, 1, d, BF, 43)
    offsets = torch.arange(0, 2 * n + 1, 2, dtype=torch.int32, device="cuda")
    x = QKV.clone()
    bad = torch.arange(0, n, 397, device="cuda")
    x[2 * bad + 1, d:] = math.nan               # the second token's key and value: the first one does not see them
    got = tp.tp_attn_core_forward(x, 1, 1, offsets=offsets)
    fine = torch.ones(2 * n, dtype=torch.bool, device="cuda")
    fine[2 * bad + 1] = False
    assert got["O"][fine].isfinite().all() and got["lse"][:, fine].isfinite().all()
    assert got["O"][~fine].isnan().all()
    some = torch.cat([bad, torch.arange(1, n, 401, device="cuda")])
    rows = torch.stack([2 * some, 2 * some + 1], 1).reshape(-1)
    O, lse, eO, el = ref.forward(QKV[rows], list(range(0, len(rows) + 1, 2)), 1, 1, 0, 0, d ** -0.5, BF)
    ok = fine[rows]
    near(got["O"][rows][ok], O[ok], eO[ok], "O")
    near(got["lse"][:, rows][:, ok], lse[:, ok], el[:, ok], "lse")
    clean = tp.tp_attn_core_forward(QKV, 1, 1, offsets=offsets)
    assert clean["O"].isfinite().all() and tp.device_status() == 0


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("window,sinks", [(10 ** 12, 3), (2 ** 32 + 7, 0), (2 ** 31, 2 ** 40)])
def test_windows_past_32_bits(window, sinks, dtype):
    gpu_or_skip()
    QKV, dO, edges, offsets = make((150, 20), 0, 2, 1, 2, 32, dtype, 44)
    check(QKV, dO, edges, offsets, 2, 1, window, sinks, dtype)
    got = tp.tp_attn_core_forward(QKV, 2, 1, offsets=offsets, window=window, sinks=sinks)
    assert torch.equal(got["O"], tp.tp_attn_core_forward(QKV, 2, 1, offsets=offsets)["O"])


def test_the_longest_sequence():
    # 2^30 tokens, a pattern of 4096 over and over: with a window all periods but the first and the last are alike
    gpu_or_skip()
    T, P, d, w = 1 << 30, 4096, 8, 33
    QKV, dO, _, _ = make((P,), 0, 0, 1, 1, d, BF, 45)
    kw = dict(n_heads=1, n_kv_heads=1, window=w)
    few = [x.repeat(4, 1) for x in (QKV, dO)]
    f = tp.tp_attn_core_forward(few[0], **kw)
    g = tp.tp_attn_core_backward(few[1], few[0], f["O"], f["lse"], **kw)
    torch.cuda.empty_cache()
    many = [x.repeat(T // P, 1) for x in (QKV, dO)]
    got = tp.tp_attn_core_forward(many[0], **kw)
    grad = tp.tp_attn_core_backward(many[1], many[0], got["O"], got["lse"], **kw)
    for x, want in ((got["O"], f["O"]), (got["lse"].T, f["lse"].T), (grad, g)):
        x, want = x.reshape(T // P, P, -1), want.reshape(4, P, -1)
        assert torch.equal(x[:2], want[:2]) and torch.equal(x[-1], want[-1])
        assert all(bool((part == want[1]).all()) for part in x[1:-1].split(1 << 14))
    assert tp.device_status() == 0
    del many, got, grad, x
    torch.cuda.empty_cache()


def test_calls_on_two_streams_at_once():
    gpu_or_skip()
    QKV, dO, _, offsets = make((700, 1300), 0, 0, 2, 4, 128, BF, 46)
    small, dsmall, _, _ = make((300,), 0, 0, 1, 2, 64, F32, 47)
    g = torch.Generator(device="cuda").manual_seed(48)
    ids = torch.randint(0, 900, (5000,), generator=g, device="cuda").int()
    dX = torch.randn(5000, 512, generator=g, device="cuda").to(BF)

    def calls(stream):
        f = tp.tp_attn_core_forward(QKV, 8, 2, offsets=offsets, window=300, sinks=4, stream=stream)
        out = [f["O"], f["lse"], tp.tp_attn_core_backward(dO, QKV, f["O"], f["lse"], 8, 2, offsets=offsets, window=300,
                                                          sinks=4, stream=stream)]
        f = tp.tp_attn_core_forward(small, 2, 1, stream=stream)
        out += [f["O"], tp.tp_attn_core_backward(dsmall, small, f["O"], f["lse"], 2, 1, stream=stream)]
        return out + [tp.tp_embedding_backward(dX, ids, 1000, stream=stream)]

    want = calls(torch.cuda.current_stream())
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(3)]
    for _ in range(10):
        for got in [calls(s) for s in streams]:
            torch.cuda.synchronize()
            assert all(torch.equal(x, y) for x, y in zip(got, want))
    assert tp.device_status() == 0
