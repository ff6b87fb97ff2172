"""Tokens sorted by expert and back against plain forms: the plan against a
sort done one assignment at a time, copies bit for bit, weighted sums and
gradients within derived bounds (_step_ref); dropped assignments, tokens
without any, experts without any, ids out of range, one token, one expert,
the most of each, places past 32 bits, another stream, a graph.

Chains: the weighted sum adds k products; a dot adds at most h / 8 products a
thread (8 to 256 threads share a token), then 5 steps over the warp and 8 over
the warps.
"""

import pytest
import torch

import vocab_ce_gb300 as tp
from _parity import gpu_or_skip
from _step_ref import D, E32, U, near
from _step_ref import plan as plain_plan

pytestmark = pytest.mark.gpu
TYPES = [torch.bfloat16, torch.float32]
# (T, k, E, share dropped): one of each, ragged, more experts than assignments, one block and several, the limits
PLANS = [(1, 1, 1, 0.0), (1, 8, 64, 0.0), (3, 2, 5, 0.5), (33, 3, 7, 0.1), (64, 32, 1024, 0.0), (100, 1, 256, 0.3),
         (999, 4, 60, 0.05), (1024, 4, 8, 0.0), (1025, 4, 8, 0.0), (5000, 8, 64, 0.1), (4099, 2, 362, 0.0),
         (200, 2, 16, 1.0), (4097, 1, 1, 0.0), (3000, 32, 1024, 0.2)]
# (T, h, k, E, share dropped): less than the fewest threads of a token, each change of their number, wide rows
ROWS = [(1, 8, 1, 1, 0.0), (5, 8, 3, 4, 0.2), (1, 4096, 2, 8, 0.0), (37, 64, 2, 5, 0.3), (300, 72, 8, 9, 0.1),
        (50, 264, 4, 16, 0.0), (129, 1000, 3, 60, 0.05), (64, 2048, 2, 8, 0.5), (70, 2056, 5, 8, 0.1),
        (33, 8192, 8, 64, 0.0), (9, 16392, 32, 40, 0.1), (40, 512, 2, 6, 1.0)]


def ids_of(T, k, E, drop, seed):
    g = torch.Generator().manual_seed(seed)
    ids = torch.randint(0, E, (T, k), generator=g, dtype=torch.int32)
    ids[torch.rand(T, k, generator=g) < drop] = -1
    if T > 4 and drop:
        ids[2] = -1                             # a token without any
    return ids


def rows(n, h, dtype, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(n, h, generator=g, device="cuda").to(dtype)


def weights_of(T, k, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(T, k, generator=g, device="cuda")


def on_gpu(plan):
    return {k: v.cuda() for k, v in plan.items()}


@pytest.mark.parametrize("T,k,E,drop", PLANS)
def test_plan(T, k, E, drop):
    gpu_or_skip()
    ids = ids_of(T, k, E, drop, T)
    want = plain_plan(ids, E)
    got = tp.tp_expert_plan(ids.cuda(), E)
    for name in ("offsets", "row", "source"):
        assert torch.equal(got[name].cpu(), want[name]), name
    assert tp.device_status() == 0


def test_plan_of_many_assignments():
    gpu_or_skip()
    T, k, E = 300_000, 8, 128
    ids = ids_of(T, k, E, 0.01, 3).cuda()
    got = tp.tp_expert_plan(ids, E)
    flat = torch.where(ids < 0, E, ids).reshape(-1)
    order = torch.sort(flat, stable=True).indices
    kept = int((ids >= 0).sum())
    assert int(got["offsets"][-1]) == kept
    assert torch.equal(got["source"][:kept].long(), order[:kept]) and bool((got["source"][kept:] == -1).all())
    assert torch.equal(got["offsets"].long().diff(), torch.bincount(flat, minlength=E + 1)[:E])
    row = got["row"].reshape(-1)
    assert torch.equal(row[order[:kept]].long(), torch.arange(kept, device="cuda"))
    assert bool((row[flat == E] == -1).all())


def test_ids_out_of_range_are_dropped_and_reported():
    gpu_or_skip()
    assert tp.device_status() == 0
    ids = torch.tensor([[0, 9], [-2, 1], [2 ** 31 - 1, -2 ** 31], [3, 8]], dtype=torch.int32)
    want = plain_plan(ids, 8)
    got = tp.tp_expert_plan(ids.cuda(), 8)
    for name, v in want.items():
        assert torch.equal(got[name].cpu(), v), name
    assert tp.device_status() == 1 and tp.device_status() == 0


def test_places_out_of_range_are_skipped_and_reported():
    # every access is guarded in the kernels: a place outside the rows is not followed
    gpu_or_skip()
    ids = ids_of(6, 2, 3, 0.0, 1)
    plan = on_gpu(plain_plan(ids, 3))
    good = {k: v.clone() for k, v in plan.items()}
    plan["row"][4, 1] = 12                      # one past the last row
    X, Ys, w = rows(6, 64, torch.float32, 1), rows(12, 64, torch.float32, 2), weights_of(6, 2, 3)
    w0 = w.clone()
    w0[4, 1] = 0.0
    assert tp.device_status() == 0
    Z = tp.tp_expert_combine_forward(Ys, plan, w)
    assert tp.device_status() == 1
    assert torch.equal(Z[:4], tp.tp_expert_combine_forward(Ys, good, w)[:4])
    near(Z[4], tp.tp_expert_combine_forward(Ys, good, w0)[4], 0.0, "skipped")
    tp.tp_expert_dispatch_forward(X, plan)
    assert tp.device_status() == 1
    got = tp.tp_expert_combine_backward(X, Ys, plan, w)
    assert tp.device_status() == 1 and got["dweights"][4, 1] == 0
    tp.tp_expert_dispatch_backward(Ys, plan)
    assert tp.device_status() == 1 and tp.device_status() == 0


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("T,h,k,E,drop", ROWS)
def test_rows(T, h, k, E, drop, dtype):
    gpu_or_skip()
    ids = ids_of(T, k, E, drop, T + h)
    cpu = plain_plan(ids, E)
    plan = on_gpu(cpu)
    n, kept = T * k, int(cpu["offsets"][-1])
    src = plan["source"][:kept].long()
    tok = src // k
    X, Ys, w = rows(T, h, dtype, 1), rows(n, h, dtype, 2), weights_of(T, k, 3)
    Ys[kept:] = float("nan")                    # rows that nobody names are not read
    dZ, dXs = rows(T, h, dtype, 4), rows(n, h, dtype, 5)
    dXs[kept:] = float("nan")

    Xs = torch.full((n, h), float("nan"), dtype=dtype, device="cuda")
    tp.tp_expert_dispatch_forward(X, plan, out=Xs)
    assert torch.equal(Xs[:kept], X[tok]) and not Xs[kept:].any()

    def back(r, wt):
        z = torch.zeros(T, h, dtype=D, device="cuda")
        return z.index_add_(0, tok, r[:kept].to(D) * (1.0 if wt is None else wt.reshape(-1)[src].to(D)[:, None]))
    Z = tp.tp_expert_combine_forward(Ys, plan, w)
    want = back(Ys, w)
    near(Z, want, U[dtype] * want.abs() + (k + 2) * E32 * back(Ys.abs(), w.abs()), "Z")
    dX = tp.tp_expert_dispatch_backward(dXs, plan)
    want = back(dXs, None)
    near(dX, want, U[dtype] * want.abs() + (k + 2) * E32 * back(dXs.abs(), None), "dX")

    out = {"dYs": torch.full((n, h), float("nan"), dtype=dtype, device="cuda")}
    got = tp.tp_expert_combine_backward(dZ, Ys, plan, w, out=out)
    assert got["dYs"] is out["dYs"] and not got["dYs"][kept:].any()
    want = dZ[tok].to(D) * w.reshape(-1)[src].to(D)[:, None]
    near(got["dYs"][:kept], want, (U[dtype] + E32) * want.abs() + 2.0 ** -130, "dYs")
    prod = dZ[tok].to(D) * Ys[:kept].to(D)
    dw, size = (torch.zeros(n, dtype=D, device="cuda") for _ in range(2))
    dw[src], size[src] = prod.sum(1), prod.abs().sum(1)
    near(got["dweights"].reshape(-1), dw, (h / 8 + 32) * E32 * size, "dweights")
    assert tp.device_status() == 0


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("k", range(1, 10))
def test_every_number_of_choices_over_many_tokens(k, dtype):
    # several vectors a thread; most choices dropped, so that most rows are only zeroed; a ragged last block
    test_rows(9001, 168, k, 16, 0.875, dtype)
    test_rows(4099, 776, k, 11, 0.0, dtype)


def test_gradients_against_differences():
    # Z is linear in each argument: a difference of any size is exact up to 64-bit roundings
    gpu_or_skip()
    T, h, k, E = 11, 72, 3, 4
    cpu = plain_plan(ids_of(T, k, E, 0.2, 7), E)
    plan, row = on_gpu(cpu), cpu["row"].long().cuda()
    Ys, w, dZ = rows(T * k, h, torch.float32, 1), weights_of(T, k, 2), rows(T, h, torch.float32, 3)
    keep = (row >= 0)[..., None]

    def f(y, ww):
        z = (torch.where(keep, y[row.clamp_min(0)], 0.0) * ww[..., None]).sum(1)
        return float((dZ.to(D) * z).sum())
    got = tp.tp_expert_combine_backward(dZ, Ys, plan, w)
    a, b = rows(T * k, h, torch.float32, 4).to(D), weights_of(T, k, 5).to(D)
    num = f(Ys.to(D) + a, w.to(D)) - f(Ys.to(D), w.to(D))
    mine = got["dYs"].to(D) * a
    assert abs(num - float(mine.sum())) <= 4 * E32 * float(mine.abs().sum())
    num = f(Ys.to(D), w.to(D) + b) - f(Ys.to(D), w.to(D))
    size = float((dZ.to(D).abs().amax() * Ys.to(D).abs().amax() * b.abs()).sum()) * h
    assert abs(num - float((got["dweights"].to(D) * b).sum())) <= (h / 8 + 32) * E32 * size


def test_no_tokens_and_refused_arguments():
    gpu_or_skip()
    got = tp.tp_expert_plan(torch.empty(0, 4, dtype=torch.int32, device="cuda"), 8)
    assert got["row"].shape == (0, 4) and got["source"].shape == (0,) and not got["offsets"].any()
    X = torch.empty(0, 64, device="cuda")
    assert tp.tp_expert_dispatch_forward(X, got).shape == (0, 64)
    assert tp.tp_expert_combine_forward(X, got, torch.empty(0, 4, device="cuda")).shape == (0, 64)
    assert tp.tp_expert_dispatch_backward(X, got).shape == (0, 64)
    assert tp.tp_expert_combine_backward(X, X, got, torch.empty(0, 4, device="cuda"))["dweights"].shape == (0, 4)
    plan = tp.tp_expert_plan(ids_of(4, 2, 3, 0.0, 1).cuda(), 3)
    with pytest.raises(ValueError, match="ids"):
        tp.tp_expert_plan(torch.zeros(4, 2, dtype=torch.int64, device="cuda"), 3)
    with pytest.raises(ValueError, match="X must"):
        tp.tp_expert_dispatch_forward(rows(5, 64, torch.float32, 1), plan)
    with pytest.raises(ValueError, match="Ys must"):
        tp.tp_expert_combine_forward(rows(4, 64, torch.float32, 1), plan, weights_of(4, 2, 1))
    with pytest.raises(ValueError, match="weights"):
        tp.tp_expert_combine_forward(rows(8, 64, torch.float32, 1), plan, weights_of(4, 3, 1))
    with pytest.raises(ValueError, match="contiguous"):
        tp.tp_expert_dispatch_forward(rows(4, 128, torch.float32, 1)[:, :64], plan)
    with pytest.raises(tp.TpceError):
        tp.tp_expert_dispatch_forward(rows(4, 20, torch.float32, 1), plan)
    with pytest.raises(tp.TpceError):
        tp.tp_expert_plan(torch.zeros(4, 33, dtype=torch.int32, device="cuda"), 40)


def test_rows_past_32_bits():
    gpu_or_skip()
    T, k, h = 65_600, 2, 16384                  # 2,149,580,800 values in the sorted rows
    ids = torch.zeros(T, k, dtype=torch.int32, device="cuda")
    ids[:, 1] = 1
    ids[-1, 0] = -1                             # the last row stays unnamed
    plan = tp.tp_expert_plan(ids, 2)
    X = torch.zeros(T, h, dtype=torch.bfloat16, device="cuda")
    X[-2:] = rows(2, h, torch.bfloat16, 1)
    Xs = tp.tp_expert_dispatch_forward(X, plan)
    n = T * k
    assert torch.equal(Xs[n - 3], X[-2]) and torch.equal(Xs[n - 2], X[-1]) and not Xs[n - 1].any()
    assert torch.equal(Xs[T - 2], X[-2]) and not Xs[T - 1].any()
    w = torch.ones(T, k, device="cuda")
    Z = tp.tp_expert_combine_forward(Xs, plan, w)
    assert torch.equal(Z[-1], X[-1]) and torch.equal(Z[-2], (2 * X[-2].float()).to(X.dtype)) and not Z[:-2].any()
    got = tp.tp_expert_combine_backward(X, Xs, plan, w)
    assert torch.equal(got["dYs"][n - 2], X[-1]) and torch.equal(got["dYs"][n - 3], X[-2])
    assert torch.equal(tp.tp_expert_dispatch_backward(Xs, plan), Z)


def test_on_another_stream_and_in_a_graph():
    gpu_or_skip()
    T, h, k, E = 200, 264, 2, 6
    ids = ids_of(T, k, E, 0.1, 5).cuda()
    X, Ys, w, dZ = (rows(T, h, torch.bfloat16, 1), rows(T * k, h, torch.bfloat16, 2), weights_of(T, k, 3),
                    rows(T, h, torch.bfloat16, 4))

    def step(stream=None, o=None):
        o = o or {}
        plan = tp.tp_expert_plan(ids, E, out=o.get("plan"), stream=stream)
        return {"plan": plan, "Xs": tp.tp_expert_dispatch_forward(X, plan, out=o.get("Xs"), stream=stream),
                "Z": tp.tp_expert_combine_forward(Ys, plan, w, out=o.get("Z"), stream=stream),
                "b": tp.tp_expert_combine_backward(dZ, Ys, plan, w, out=o.get("b"), stream=stream),
                "dX": tp.tp_expert_dispatch_backward(Ys, plan, out=o.get("dX"), stream=stream)}

    def same(a, b):
        for key in a:
            for x, y in zip(a[key].values(), b[key].values()) if isinstance(a[key], dict) else [(a[key], b[key])]:
                assert torch.equal(x, y), key
    ref = step()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = step(side)
    torch.cuda.current_stream().wait_stream(side)
    same(ref, got)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(o=got)
    ids.copy_(ids_of(T, k, E, 0.3, 6))
    graph.replay()
    same(step(), got)
    assert tp.device_status() == 0
