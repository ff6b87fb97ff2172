"""The embedding and its gradient against 64-bit forms: rows by id bit for bit
where the scale is a power of two, sums within derived bounds (_step_ref);
padding, ids out of range, one token, one id for all tokens (a run over every
chunk), tables of one to three sorting passes, one block and several, rows past
32 bits, tables that are added to, another stream, a graph.

Chains: a run of c equal ids adds c rows, then (where it crosses chunks) at most
c more partial sums, the scale's product and the old value.
"""

import math

import pytest
import torch

import vocab_ce_gb300 as tp
from _parity import gpu_or_skip
from _step_ref import D, E32, U, near

pytestmark = pytest.mark.gpu
TYPES = [torch.bfloat16, torch.float32]
# (T, h, v_pad, v_valid, kind of ids)
CASES = [(1, 8, 1, 1, "random"), (1, 8192, 128, 100, "random"), (3, 64, 5, 5, "same"), (17, 72, 128, 128, "random"),
         (16, 1000, 64, 60, "random"), (33, 2056, 640, 600, "zipf"), (100, 520, 300, 300, "none"),
         (999, 1000, 1024, 1000, "zipf"), (1000, 264, 2048, 2000, "same"), (2048, 24, 1023, 1023, "zipf"),
         (2049, 24, 1024, 1024, "zipf"), (5000, 4096, 1280, 1200, "zipf"), (4100, 128, 50304, 50257, "padded"),
         (3000, 8, (1 << 20) + 7, (1 << 20) + 1, "random"), (3000, 16, 1 << 20, 1 << 20, "sorted"),
         (1500, 8, (1 << 21) + 3, (1 << 21) + 3, "random"), (300_000, 8, 5000, 5000, "zipf"),
         (20_000, 40, 64, 64, "same")]


def ids_of(T, v, kind, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    if kind == "same":
        ids = torch.full((T,), v - 1, device="cuda")
    elif kind == "none":
        ids = torch.full((T,), -1, device="cuda")
    elif kind == "zipf":
        u = torch.rand(T, generator=g, device="cuda", dtype=D)
        ids = ((v + 1.0) ** u).floor().clamp(1, v) - 1
    else:
        ids = torch.randint(0, v, (T,), generator=g, device="cuda")
    if kind == "sorted":
        ids = ids.sort().values
    if kind in ("zipf", "padded"):
        ids = torch.where(torch.rand(T, generator=g, device="cuda") < (0.4 if kind == "padded" else 0.05), -1, ids)
    return ids.int()


def rows(n, h, dtype, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(n, h, generator=g, device="cuda").to(dtype)


def sums(dX, ids, v_pad):
    """The runs' sums and the sums of their absolute values in 64 bits, and the runs' lengths."""
    kept = ids >= 0
    at = ids[kept].long()
    x = dX[kept].to(D)
    zero = torch.zeros(v_pad, dX.shape[1], dtype=D, device="cuda")
    return zero.index_add(0, at, x), zero.index_add(0, at, x.abs()), torch.bincount(at, minlength=v_pad)


def check_backward(got, dX, ids, v_pad, scale, dtype, old=None):
    scale = torch.tensor(scale, dtype=torch.float32).to(D).item()
    want, size, runs = sums(dX, ids, v_pad)
    want, size = want * scale, size * abs(scale)
    chain = (2 * runs + 2).to(D)[:, None]
    if old is not None:
        want, size = want + old.to(D), size + old.to(D).abs()
    err = chain * E32 * size
    near(got, want, err + U[dtype] * (want.abs() + err), "dE")
    return runs


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("T,h,v_pad,v_valid,kind", CASES)
def test_rows_and_gradient(T, h, v_pad, v_valid, kind, dtype):
    gpu_or_skip()
    ids = ids_of(T, v_valid, kind, T + h)
    E, dX = rows(v_pad, h, dtype, 1), rows(T, h, dtype, 2)
    want = torch.where(ids[:, None] >= 0, E[ids.clamp_min(0).long()], 0.0)
    assert torch.equal(tp.tp_embedding_forward(ids, E, v_valid=v_valid), want)
    assert torch.equal(tp.tp_embedding_forward(ids, E, v_valid=v_valid, scale=-0.5).float(), want.float() * -0.5)
    scale = torch.tensor(math.sqrt(h + 1.0), dtype=torch.float32).item()
    w = want.to(D) * scale
    near(tp.tp_embedding_forward(ids, E, v_valid=v_valid, scale=scale), w,
         (E32 + U[dtype] * (1 + E32)) * w.abs(), "X")      # the product's rounding and the stored one
    dE = tp.tp_embedding_backward(dX, ids, v_pad, v_valid=v_valid, scale=scale)
    runs = check_backward(dE, dX, ids, v_pad, scale, dtype)
    assert not dE[runs == 0].float().any()
    again = tp.tp_embedding_backward(dX, ids, v_pad, v_valid=v_valid, scale=scale)
    assert torch.equal(dE, again)
    # added to a table whose other rows hold what must not be touched
    old = rows(v_pad, h, dtype, 3)
    old[runs == 0] = math.nan
    new = old.clone()
    assert tp.tp_embedding_backward(dX, ids, v_pad, v_valid=v_valid, scale=scale, out=new, accumulate=True) is new
    named = runs > 0
    assert torch.equal(new[~named].view(torch.uint8), old[~named].view(torch.uint8))
    got = torch.where(named[:, None], new, 0.0)
    check_backward(got, dX, ids, v_pad, scale, dtype, torch.where(named[:, None], old, 0.0))
    assert tp.device_status() == 0


def test_gradient_against_differences():
    # the loss sum(W X) is linear in E: differences are exact up to rounding
    gpu_or_skip()
    T, h, v = 50, 16, 12
    ids = ids_of(T, v, "zipf", 5)
    E, W = rows(v, h, torch.float32, 6), rows(T, h, torch.float32, 7)
    dE = tp.tp_embedding_backward(W, ids, v, scale=3.0)
    for r, c in [(0, 0), (1, 7), (4, 15), (11, 3)]:
        up, down = E.clone(), E.clone()
        up[r, c] += 1.0
        down[r, c] -= 1.0
        x = [(tp.tp_embedding_forward(ids, e, scale=3.0).to(D) * W.to(D)).sum() for e in (up, down)]
        # both tables' values and products are rounded: 2 T terms of |E| + 1, times 3 |W|
        tol = 6 * E32 * 3 * (W.abs()[:, c].sum() * (E.abs().max() + 1)).item()
        assert abs(((x[0] - x[1]) / 2 - dE[r, c].to(D)).item()) <= tol


def test_ids_out_of_range_are_padding_and_reported():
    gpu_or_skip()
    assert tp.device_status() == 0
    v_pad, v_valid, h = 128, 100, 64
    bad = torch.tensor([5, 100, 127, 128, -2, 2 ** 31 - 1, -2 ** 31, 99, 5], dtype=torch.int32, device="cuda")
    good = torch.tensor([5, -1, -1, -1, -1, -1, -1, 99, 5], dtype=torch.int32, device="cuda")
    E, dX = rows(v_pad, h, torch.bfloat16, 1), rows(9, h, torch.bfloat16, 2)
    X = tp.tp_embedding_forward(bad, E, v_valid=v_valid)
    assert tp.device_status() == 1
    assert torch.equal(X, tp.tp_embedding_forward(good, E, v_valid=v_valid))
    dE = tp.tp_embedding_backward(dX, bad, v_pad, v_valid=v_valid)
    assert tp.device_status() == 1
    assert torch.equal(dE, tp.tp_embedding_backward(dX, good, v_pad, v_valid=v_valid))
    assert tp.device_status() == 0


def test_infinities_and_nan_stay_in_their_rows():
    gpu_or_skip()
    ids = torch.tensor([3, 1, 3, 0, 1, -1, 2], dtype=torch.int32, device="cuda")
    dX = rows(7, 64, torch.bfloat16, 1)
    dX[1, 5], dX[4, 5], dX[0, 6], dX[5] = math.inf, -math.inf, math.inf, math.nan
    dE = tp.tp_embedding_backward(dX, ids, 8).float()
    assert dE[1, 5].isnan() and dE[3, 6] == math.inf and int((~dE.isfinite()).sum()) == 2
    E = rows(8, 64, torch.float32, 2)
    E[4:] = math.nan
    assert bool(tp.tp_embedding_forward(ids, E).isfinite().all())


def test_no_tokens():
    gpu_or_skip()
    ids = torch.empty(0, dtype=torch.int32, device="cuda")
    X = tp.tp_embedding_forward(ids, rows(8, 64, torch.float32, 1))
    assert X.shape == (0, 64)
    dE = torch.full((8, 64), 3.0, device="cuda")
    assert tp.tp_embedding_backward(X, ids, 8, out=dE, accumulate=True) is dE and bool((dE == 3.0).all())
    assert not tp.tp_embedding_backward(X, ids, 8, out=dE).any()


def test_table_past_32_bits():
    gpu_or_skip()
    h = 8192
    v = (1 << 31) // h + 65                       # values past 2^31 from row 262,144 on
    E = torch.zeros(v, h, dtype=torch.bfloat16, device="cuda")
    ids = torch.tensor([v - 1, 0, (1 << 31) // h, v - 1], dtype=torch.int32, device="cuda")
    dX = rows(4, h, torch.bfloat16, 1)
    E[ids[:3].long()] = dX[:3]
    assert torch.equal(tp.tp_embedding_forward(ids, E)[:3], dX[:3])
    assert tp.tp_embedding_backward(dX, ids, v, out=E) is E
    want = {v - 1: (dX[0].float() + dX[3].float()).to(torch.bfloat16), 0: dX[1], (1 << 31) // h: dX[2]}
    for r, x in want.items():
        assert torch.equal(E[r], x)
        E[r] = 0
    assert not any(bool(E[i:i + 32768].any()) for i in range(0, v, 32768))


def test_another_stream_and_a_given_workspace():
    gpu_or_skip()
    T, h, v = 3000, 256, 500
    ids, dX, E = ids_of(T, v, "zipf", 1), rows(T, h, torch.bfloat16, 2), rows(v, h, torch.bfloat16, 3)
    want, grad = tp.tp_embedding_forward(ids, E), tp.tp_embedding_backward(dX, ids, v)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    ws = torch.full((tp.embedding_workspace_bytes(T, h, v),), 0xff, dtype=torch.uint8, device="cuda")
    s.wait_stream(torch.cuda.current_stream())
    X = tp.tp_embedding_forward(ids, E, stream=s)
    dE = tp.tp_embedding_backward(dX, ids, v, ws=ws, stream=s)
    s.synchronize()
    assert torch.equal(X, want) and torch.equal(dE, grad)


def test_in_a_graph():
    gpu_or_skip()
    T, h, v = 2500, 128, 700
    ids, dX, E = ids_of(T, v, "zipf", 1), rows(T, h, torch.bfloat16, 2), rows(v, h, torch.bfloat16, 3)
    X, dE = torch.empty(T, h, dtype=E.dtype, device="cuda"), torch.zeros_like(E)
    ws = torch.empty(tp.embedding_workspace_bytes(T, h, v), dtype=torch.uint8, device="cuda")

    def step():
        tp.tp_embedding_forward(ids, E, out=X)
        tp.tp_embedding_backward(dX, ids, v, out=dE, accumulate=True, ws=ws)

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
    torch.cuda.current_stream().wait_stream(s)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for seed in (4, 5):
        ids.copy_(ids_of(T, v, "zipf", seed))
        dX.copy_(rows(T, h, torch.bfloat16, seed))
        old = rows(v, h, torch.bfloat16, seed + 10)
        dE.copy_(old)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(X, tp.tp_embedding_forward(ids, E))
        assert torch.equal(dE, tp.tp_embedding_backward(dX, ids, v, out=old, accumulate=True))


def test_what_is_written_counts_as_changed():
    gpu_or_skip()
    ids, dX = ids_of(10, 8, "random", 1), rows(10, 64, torch.float32, 2)
    out, X = torch.zeros(8, 64, device="cuda"), torch.empty(10, 64, device="cuda")
    tp.tp_embedding_backward(dX, ids, 8, out=out, accumulate=True)
    tp.tp_embedding_forward(ids, out, out=X)
    assert (out._version, X._version, dX._version, ids._version) == (1, 1, 0, 0)


def test_tensors_that_are_refused():
    gpu_or_skip()
    ids, E = ids_of(10, 8, "random", 1), rows(8, 64, torch.float32, 2)
    dX = rows(10, 64, torch.float32, 3)
    for bad in (ids.long(), ids.cpu(), ids.reshape(2, 5), ids.repeat_interleave(2)[::2]):
        with pytest.raises(ValueError):
            tp.tp_embedding_forward(bad, E)
        with pytest.raises(ValueError):
            tp.tp_embedding_backward(dX, bad, 8)
    for bad in (E.half(), E.cpu(), E.T, E[0]):
        with pytest.raises(ValueError):
            tp.tp_embedding_forward(ids, bad)
    with pytest.raises(ValueError, match="accumulate"):
        tp.tp_embedding_backward(dX, ids, 8, accumulate=True)
    with pytest.raises(ValueError):
        tp.tp_embedding_backward(dX, ids, 8, out=E[:7])
    with pytest.raises(ValueError):
        tp.tp_embedding_backward(dX, ids, 8, out=E.bfloat16())
    with pytest.raises(ValueError):
        tp.tp_embedding_backward(dX, ids, 0)
    for kw in ({"v_valid": 9}, {"v_valid": 0}, {"scale": math.inf}, {"scale": math.nan}):
        with pytest.raises(tp.TpceError):
            tp.tp_embedding_forward(ids, E, **kw)
        with pytest.raises(tp.TpceError):
            tp.tp_embedding_backward(dX, ids, 8, **kw)
    big = rows(18, 64, torch.float32, 4)
    with pytest.raises(tp.TpceError, match="overlap"):
        tp.tp_embedding_backward(big[:10], ids, 9, out=big[9:])
    with pytest.raises(tp.TpceError, match="overlap"):
        tp.tp_embedding_forward(ids, big[:8], out=big[7:17])


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("T,h,v_pad", [
    (70_000, 8, 90_001), (70_000, 64, 5000), (66_000, 1000, 3001),  # more tokens than a cluster sorts
    (66_000, 5000, 401),
    (5, 1024, 60_000), (200, 16, 4_000_000),                        # larger tables than it zeroes
    (900, 1000, 30_001),
])
def test_every_row_of_a_new_table_is_written(T, h, v_pad, dtype):
    gpu_or_skip()
    ids, dX = ids_of(T, v_pad, "zipf", 21), rows(T, h, dtype, 22)
    dE = torch.full((v_pad, h), math.nan, device="cuda", dtype=dtype)
    tp.tp_embedding_backward(dX, ids, v_pad, out=dE)
    runs = torch.bincount(ids[ids >= 0].long(), minlength=v_pad)
    assert not dE[runs == 0].view(torch.uint8).any()
    named = (runs > 0).nonzero()[:, 0]
    at = torch.full((v_pad,), -1, dtype=torch.int32, device="cuda")
    at[named] = torch.arange(len(named), dtype=torch.int32, device="cuda")
    few = torch.where(ids >= 0, at[ids.clamp_min(0).long()], -1)
    check_backward(dE[named], dX, few, len(named), 1.0, dtype)
    assert tp.device_status() == 0


@pytest.mark.parametrize("T", [1, 31, 32, 33, 1000, 2047, 2048, 2049, 4064, 4095, 4096, 4097])
@pytest.mark.parametrize("v_pad", [7, 50_000, (1 << 24) - 1, 1 << 24])
def test_lengths_around_the_kinds_of_sorts(T, v_pad):
    # whole numbers: sums are exact in any split, and a token in another's place would be seen
    gpu_or_skip()
    for kind in ("random", "zipf", "same", "sorted"):
        ids = ids_of(T, v_pad, kind, T)
        dX = torch.arange(T, device="cuda", dtype=torch.float32)[:, None].expand(T, 8).contiguous() % 1024
        # places that no token was sorted to would name row 0
        ws = torch.zeros(tp.embedding_workspace_bytes(T, 8, v_pad), dtype=torch.uint8, device="cuda")
        dE = tp.tp_embedding_backward(dX, ids, v_pad, ws=ws)
        want = torch.zeros(v_pad, 8, device="cuda").index_add_(0, ids.clamp_min(0).long(),
                                                              torch.where(ids[:, None] >= 0, dX, 0.0))
        assert torch.equal(dE, want), kind
        dX = rows(T, 8, torch.float32, 5)
        assert torch.equal(tp.tp_embedding_backward(dX, ids, v_pad), tp.tp_embedding_backward(dX, ids, v_pad)), kind
    assert tp.device_status() == 0


def test_ids_that_are_part_of_a_batch():
    # inputs and targets of next-token prediction are the same rows, one token apart: not 16-byte aligned
    gpu_or_skip()
    v, h, T = 500, 64, 99
    tokens = ids_of(3 * (T + 1), v, "zipf", 31).reshape(3, T + 1)
    E, dX = rows(v, h, torch.bfloat16, 32), rows(T, h, torch.bfloat16, 33)
    for b in range(3):
        for ids in (tokens[b, :-1], tokens[b, 1:], tokens[b, 3:]):
            n = len(ids)
            X, dE = tp.tp_embedding_forward(ids.clone(), E), tp.tp_embedding_backward(dX[:n], ids.clone(), v)
            assert torch.equal(tp.tp_embedding_forward(ids, E), X)
            assert torch.equal(tp.tp_embedding_backward(dX[:n], ids, v), dE)
            s = torch.cuda.Stream()
            s.wait_stream(torch.cuda.current_stream())
            other = tp.tp_embedding_forward(ids, E, stream=s), tp.tp_embedding_backward(dX[:n], ids, v, stream=s)
            s.synchronize()
            assert torch.equal(other[0], X) and torch.equal(other[1], dE)
    # captured: what the tokens are at the replay counts
    ids, X, dE = tokens[1, 1:], torch.empty_like(dX), torch.empty_like(E)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        tp.tp_embedding_forward(ids, E, out=X)
        tp.tp_embedding_backward(dX, ids, v, out=dE)
    for seed in (34, 35):
        tokens.copy_(ids_of(3 * (T + 1), v, "zipf", seed).reshape(3, T + 1))
        g.replay()
        assert torch.equal(X, tp.tp_embedding_forward(ids.clone(), E))
        assert torch.equal(dE, tp.tp_embedding_backward(dX, ids.clone(), v))
    assert tp.device_status() == 0


@pytest.mark.parametrize("T", [4097, 5000, 65_536, 65_537, 70_000, 300_000])
@pytest.mark.parametrize("v_pad", [1 << 20, (1 << 20) + 7, (1 << 21) + 3])
def test_three_passes_of_a_sort(T, v_pad):
    # 2^20 keys and the one for padding no longer fit two passes of ten bits; each token's row is its number's
    # digits, whose sums are exact in any split, and which tell one token from another
    gpu_or_skip()
    t = torch.arange(T, device="cuda")
    dX = torch.stack([t >> 4 * c & 15 for c in range(8)], 1).float()
    for kind in ("random", "zipf", "same", "sorted"):
        ids = ids_of(T, v_pad, kind, T)
        ids[::7] = v_pad - 1                    # the largest key
        want = torch.zeros(v_pad, 8, device="cuda").index_add_(0, ids.clamp_min(0).long(),
                                                              torch.where(ids[:, None] >= 0, dX, 0.0))
        assert float(want.max()) < 2 ** 24
        ws = torch.zeros(tp.embedding_workspace_bytes(T, 8, v_pad), dtype=torch.uint8, device="cuda")
        assert torch.equal(tp.tp_embedding_backward(dX, ids, v_pad, ws=ws), want), kind
    assert tp.device_status() == 0


@pytest.mark.parametrize("T", [3000, 5000, 70_000])
def test_the_largest_table(T):
    # 2^30 rows: ids of 31 bits, in four passes
    gpu_or_skip()
    v, h = 1 << 30, 8
    ids = ids_of(T, v, "random", T)
    ids[::5], ids[1::5], ids[2::11] = v - 1, 7, -1
    dX = (torch.arange(T * h, device="cuda").reshape(T, h) % 4).to(torch.bfloat16)
    kept = ids >= 0
    named, at = ids[kept].long().unique(return_inverse=True)
    want = torch.zeros(len(named), h, device="cuda").index_add_(0, at, dX[kept].float()).to(torch.bfloat16)
    dE = tp.tp_embedding_backward(dX, ids, v)
    assert torch.equal(dE[named], want)
    X = torch.where(kept[:, None], dE[ids.clamp_min(0).long()], 0.0)
    assert torch.equal(tp.tp_embedding_forward(ids, dE), X)
    dE[named] = 0
    assert not any(bool(part.view(torch.int16).any()) for part in dE.split(1 << 27))
    assert tp.device_status() == 0
