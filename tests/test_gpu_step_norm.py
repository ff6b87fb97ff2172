"""RMS norm with the residual's addition against the plain 64-bit form: widths
and row counts on both sides of every change of layout, 8-bit outputs, rows
that hold nothing or infinities, in-place calls, another stream, gradients
against the formula and against differences. Bounds: _step_ref.

Chains: a thread adds up to 32 squares one after the other, then 5 + 5 steps
over the warp and the block, so 45 roundings at most; 64 allows for the mean,
the root and the products as well. dw: at least 152 blocks share the rows (or
each has one), so a block adds T / 152 of them one after the other at most;
then up to 32 of a block's rows and the blocks' partial rows, in chains of 32,
38 and 32.
"""

import pytest
import torch

import vocab_ce_gb300 as tp
from _parity import gpu_or_skip
from _step_ref import D, E32, U, codes_near, group_scale, near, norm_backward, norm_forward

pytestmark = pytest.mark.gpu
EPS = 1e-6
C = 64 * E32
TYPES = [torch.bfloat16, torch.float32]
# one row, rows of 8, 16 and 32 lanes and a block's first ones, a group's edge, 1, 2 and 4 vectors a thread, with
# and without more rows than blocks, the widest
SHAPES = [(1, 8), (3, 64), (1000, 120), (5, 128), (9, 136), (17, 256), (700, 264), (33, 512), (4, 1000), (65, 1024),
          (1, 1032), (641, 1032), (7, 2048), (3, 4096), (2, 4104), (611, 8192), (5, 8200), (3, 16384), (306, 16376)]


def rows(T, h, dtype, seed, std=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (std * torch.randn(T, h, generator=g, device="cuda")).to(dtype)


def weight(h, seed=9):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return 1.0 + 0.2 * torch.randn(h, generator=g, device="cuda")


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("T,h", SHAPES)
@pytest.mark.parametrize("residual", [False, True])
def test_forward(T, h, dtype, residual):
    gpu_or_skip()
    X, w = rows(T, h, dtype, 1), weight(h)
    R = rows(T, h, dtype, 2, 3.0) if residual else None
    got = tp.tp_rmsnorm_forward(X, w, R, eps=EPS, quantize=True)
    S = X
    if residual:
        S = (X.float() + R.float()).to(dtype)
        assert torch.equal(got["S"], S)
    Y, rstd = norm_forward(S, w, EPS)
    near(got["rstd"], rstd, C * rstd, "rstd")
    near(got["Y"], Y, (U[dtype] + C) * Y.abs() + 2.0 ** -130, "Y")
    codes_near(got["Q"], got["Q_scale"], Y, C * Y.abs() + 2.0 ** -130, "Q")
    # without the 8-bit output, and without the other one, the same bits
    assert torch.equal(tp.tp_rmsnorm_forward(X, w, R, eps=EPS)["Y"], got["Y"])
    only = tp.tp_rmsnorm_forward(X, w, R, eps=EPS, quantize=True, want_Y=False)
    assert "Y" not in only and torch.equal(only["Q"].view(torch.uint8), got["Q"].view(torch.uint8))
    assert torch.equal(only["Q_scale"], got["Q_scale"])


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("h", [1024, 2040, 2048, 4080, 4096, 6136, 6144, 12288])
@pytest.mark.parametrize("residual", [False, True])
def test_forward_whose_rows_in_flight_are_just_48_kb(h, dtype, residual):
    # more shared memory than a launch gets without asking begins there, with what the kernel declares counted in
    test_forward(1500, h, dtype, residual)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("T,h", SHAPES)
@pytest.mark.parametrize("residual", [False, True])
def test_backward(T, h, dtype, residual):
    gpu_or_skip()
    S, dY, w = rows(T, h, dtype, 3), rows(T, h, dtype, 4), weight(h)
    dS = rows(T, h, dtype, 5) if residual else None
    rstd = norm_forward(S, w, EPS)[1].float()
    got = tp.tp_rmsnorm_backward(dY, S, w, rstd, dS)
    dX, dw = norm_backward(dY, S, w, EPS, dS)
    r, g = rstd.to(D)[:, None], (dY.to(D) * w.to(D)).abs()
    xh = S.to(D).abs() * r
    size = r * (g + xh * (g * xh).mean(-1, keepdim=True)) + (0 if dS is None else dS.to(D).abs())
    near(got["dX"], dX, U[dtype] * dX.abs() + 2 * C * size, "dX")
    near(got["dw"], dw, (128 + T / 152) * E32 * (dY.to(D).abs() * xh).sum(0), "dw")
    # the same call again: the same bits; without dw too
    again = tp.tp_rmsnorm_backward(dY, S, w, rstd, dS)
    assert torch.equal(again["dX"], got["dX"]) and torch.equal(again["dw"], got["dw"])
    alone = tp.tp_rmsnorm_backward(dY, S, w, rstd, dS, want_dw=False)
    assert "dw" not in alone and torch.equal(alone["dX"], got["dX"])


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("T,h", [(1, 8208), (75, 16384), (77, 8200), (152, 8208), (380, 12288), (1003, 8200), (1003, 16384)])
@pytest.mark.parametrize("residual", [False, True])
def test_backward_of_rows_that_two_blocks_share(T, h, dtype, residual):
    # 76 pairs of blocks: fewer rows than pairs, as many as the ring's stages, many times those; halves of different
    # lengths. A pair adds T / 76 rows to dw one after the other. In place, on a stream of its own, and a row
    # that holds an infinity beside rows that do not.
    gpu_or_skip()
    S, dY, w = rows(T, h, dtype, 3), rows(T, h, dtype, 4), weight(h)
    dS = rows(T, h, dtype, 5) if residual else None
    rstd = norm_forward(S, w, EPS)[1].float()
    got = tp.tp_rmsnorm_backward(dY, S, w, rstd, dS)
    dX, dw = norm_backward(dY, S, w, EPS, dS)
    r, g = rstd.to(D)[:, None], (dY.to(D) * w.to(D)).abs()
    xh = S.to(D).abs() * r
    size = r * (g + xh * (g * xh).mean(-1, keepdim=True)) + (0 if dS is None else dS.to(D).abs())
    near(got["dX"], dX, U[dtype] * dX.abs() + 2 * C * size, "dX")
    near(got["dw"], dw, (128 + T / 76) * E32 * (dY.to(D).abs() * xh).sum(0), "dw")
    a = [dY.clone()] + ([dS.clone()] if residual else [])
    side = torch.cuda.Stream()
    for into in a:
        side.wait_stream(torch.cuda.current_stream())
        again = tp.tp_rmsnorm_backward(a[0], S, w, rstd, a[1] if residual else None, out={"dX": into}, stream=side)
        torch.cuda.current_stream().wait_stream(side)
        assert torch.equal(into, got["dX"]) and torch.equal(again["dw"], got["dw"])
        a[0].copy_(dY)
    last = dY.clone()
    last[T - 1, h - 1] = float("inf")
    odd = tp.tp_rmsnorm_backward(last, S, w, rstd, dS, want_dw=False)["dX"]
    assert torch.equal(odd[:T - 1], got["dX"][:T - 1]) and not bool(odd[T - 1].isfinite().any())


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("T,h", [(32767, 264), (32768, 264), (40_001, 512), (33_000, 1024)])
def test_backward_of_many_rows(T, h, dtype):
    test_backward(T, h, dtype, True)


def test_gradient_against_differences():
    # f = sum dY Y over the plain 64-bit forward; central differences in 64 bits with step 1e-5 are off by
    # about 1e-10 of f's third derivative, far below the kernel's own fp32 error
    gpu_or_skip()
    T, h = 5, 264
    S, dY, w = rows(T, h, torch.float32, 6), rows(T, h, torch.float32, 7), weight(h)
    got = tp.tp_rmsnorm_backward(dY, S, w, tp.tp_rmsnorm_forward(S, w, eps=EPS)["rstd"])

    def f(x, ww):
        return float((dY.to(D) * norm_forward(x, ww, EPS)[0]).sum())
    d = 1e-5
    for seed in range(4):
        v = rows(T, h, torch.float32, 20 + seed).to(D)
        num = (f(S.to(D) + d * v, w) - f(S.to(D) - d * v, w)) / (2 * d)
        mine = float((got["dX"].to(D) * v).sum())
        assert abs(num - mine) <= 4 * C * float((got["dX"].to(D) * v).abs().sum() + h), (num, mine)
        u = rows(1, h, torch.float32, 40 + seed).to(D)[0]
        num = (f(S, w.to(D) + d * u) - f(S, w.to(D) - d * u)) / (2 * d)
        mine = float((got["dw"].to(D) * u).sum())
        size = float((dY.to(D).abs() * norm_forward(S, w, EPS)[0].abs() / w.to(D).abs() * u.abs()).sum())
        assert abs(num - mine) <= 4 * C * size, (num, mine)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("h", [264, 2048])
def test_rows_of_zeros_and_of_infinities(dtype, h):
    gpu_or_skip()
    X, w = rows(6, h, dtype, 8), weight(h)
    X[1] = 0.0
    X[2, 5] = float("inf")
    X[3, 7] = float("nan")
    X[4] = 1e30                                  # squares that leave fp32
    got = tp.tp_rmsnorm_forward(X, w, eps=EPS, quantize=True)
    Y = got["Y"]
    assert not Y[1].any() and not got["Q"][1].float().any() and bool((got["Q_scale"][1] == 2.0 ** -126).all())
    # an infinity's row has rstd 0: zeros, and NaN where the infinity is
    assert got["rstd"][2] == 0 and Y[2, 5].isnan() and not Y[2, :5].any() and not Y[2, 6:].any()
    assert got["Q"][2, 5].float().isnan() and not got["Q"][2, 6:].float().any()
    assert bool(Y[3].isnan().all()) and bool(got["Q"][3].float().isnan().all())
    assert bool((got["Q_scale"][3] == 2.0 ** -126).all())
    assert got["rstd"][4] == 0 and not Y[4].any()
    # the rows beside them are untouched by their neighbours
    for r in (0, 5):
        y, _ = norm_forward(X[r:r + 1], w, EPS)
        near(Y[r:r + 1], y, (U[dtype] + C) * y.abs(), f"row {r}")


def test_eight_bit_codes_saturate_nothing_and_mark_what_is_not_finite():
    # weights make single values infinite: the group keeps its finite values' scale
    gpu_or_skip()
    X, w = rows(2, 1040, torch.float32, 10), weight(1040)
    w[3], w[200] = float("inf"), float("nan")
    got = tp.tp_rmsnorm_forward(X, w, eps=EPS, quantize=True)
    q = got["Q"].float()
    assert bool(q[:, 3].isnan().all()) and bool(q[:, 200].isnan().all())
    fine = torch.ones(1040, dtype=torch.bool, device="cuda")
    fine[3] = fine[200] = False
    assert bool(q[:, fine].isfinite().all())
    near(got["Q_scale"], group_scale(got["Y"]), C * got["Q_scale"].to(D), "scale")
    assert float(q[:, fine].abs().amax()) == 448.0


def test_in_place_and_on_another_stream():
    gpu_or_skip()
    T, h = 300, 1032
    X, R, w = rows(T, h, torch.bfloat16, 11), rows(T, h, torch.bfloat16, 12), weight(h)
    ref = tp.tp_rmsnorm_forward(X, w, R)
    into = R.clone()
    got = tp.tp_rmsnorm_forward(X, w, into, out={"S": into})
    assert got["S"] is into and torch.equal(into, ref["S"]) and torch.equal(got["Y"], ref["Y"])
    into = X.clone()
    got = tp.tp_rmsnorm_forward(into, w, R, out={"S": into})
    assert torch.equal(into, ref["S"]) and torch.equal(got["Y"], ref["Y"])
    dY, dS = rows(T, h, torch.bfloat16, 13), rows(T, h, torch.bfloat16, 14)
    b = tp.tp_rmsnorm_backward(dY, ref["S"], w, ref["rstd"], dS)
    for which in (0, 1):
        a = [dY.clone(), dS.clone()]
        got = tp.tp_rmsnorm_backward(a[0], ref["S"], w, ref["rstd"], a[1], out={"dX": a[which]})
        assert got["dX"] is a[which] and torch.equal(a[which], b["dX"]) and torch.equal(got["dw"], b["dw"])
    side = torch.cuda.Stream()
    for _ in range(3):
        side.wait_stream(torch.cuda.current_stream())
        f = tp.tp_rmsnorm_forward(X, w, R, quantize=True, stream=side)
        c = tp.tp_rmsnorm_backward(dY, f["S"], w, f["rstd"], dS, stream=side)
        torch.cuda.current_stream().wait_stream(side)
        assert torch.equal(f["Y"], ref["Y"]) and torch.equal(c["dX"], b["dX"]) and torch.equal(c["dw"], b["dw"])


def test_no_rows_and_refused_arguments():
    gpu_or_skip()
    w = weight(64)
    X = torch.empty(0, 64, dtype=torch.bfloat16, device="cuda")
    got = tp.tp_rmsnorm_forward(X, w, X, quantize=True)
    assert got["Y"].shape == (0, 64) and got["Q_scale"].shape == (0, 1)
    b = tp.tp_rmsnorm_backward(X, X, w, got["rstd"], X)
    assert b["dX"].shape == (0, 64) and not b["dw"].any()
    Y = rows(4, 128, torch.bfloat16, 1)
    with pytest.raises(ValueError, match="contiguous"):
        tp.tp_rmsnorm_forward(Y[:, :64], w)
    with pytest.raises(ValueError, match="w must"):
        tp.tp_rmsnorm_forward(Y, w)
    with pytest.raises(ValueError, match="want_Y"):
        tp.tp_rmsnorm_forward(rows(4, 64, torch.bfloat16, 1), w, want_Y=False)
    with pytest.raises(ValueError, match="S must"):
        tp.tp_rmsnorm_forward(Y, weight(128), Y, out={"S": torch.empty(3, 128, dtype=Y.dtype, device="cuda")})
    with pytest.raises(tp.TpceError):
        tp.tp_rmsnorm_forward(rows(2, 20, torch.float32, 1), weight(20))
    with pytest.raises(tp.TpceError):          # a start that is not on 16 bytes
        tp.tp_rmsnorm_forward(rows(1, 72, torch.bfloat16, 1).reshape(-1)[4:68].reshape(1, 64), w)


def test_more_values_than_32_bits_count():
    gpu_or_skip()
    T, h = 131_080, 16384                       # 2,147,614,720 values
    X, w = torch.zeros(T, h, dtype=torch.bfloat16, device="cuda"), weight(h)
    X[-3:] = rows(3, h, torch.bfloat16, 15)
    got = tp.tp_rmsnorm_forward(X, w, eps=EPS, quantize=True)
    Y, rstd = norm_forward(X[-3:], w, EPS)
    near(got["Y"][-3:], Y, (U[X.dtype] + C) * Y.abs(), "Y")
    codes_near(got["Q"][-3:], got["Q_scale"][-3:], Y, C * Y.abs(), "Q")
    assert not got["Y"][:64].any() and not got["Y"][-67:-3].any()
    dY = X                                      # zeros, and the same three rows
    b = tp.tp_rmsnorm_backward(dY, X, w, got["rstd"])
    dX, dw = norm_backward(X[-3:], X[-3:], w, EPS)
    size = rstd[:, None] * X[-3:].to(D).abs() * 4 * (1 + w.to(D).abs()) * X[-3:].to(D).abs().amax()
    near(b["dX"][-3:], dX, U[X.dtype] * dX.abs() + 2 * C * size, "dX")
    near(b["dw"], dw, 128 * E32 * (X[-3:].to(D).pow(2) * rstd[:, None]).sum(0) + 2.0 ** -130, "dw")


def test_captured_into_a_graph():
    gpu_or_skip()
    T, h = 70, 2048
    X, R, dY, w = *(rows(T, h, torch.bfloat16, s) for s in (16, 17, 18)), weight(h)
    out = tp.tp_rmsnorm_forward(X, w, R, quantize=True)
    back = tp.tp_rmsnorm_backward(dY, out["S"], w, out["rstd"])
    ws = torch.empty(tp.rmsnorm_workspace_bytes(T, h), dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        tp.tp_rmsnorm_forward(X, w, R, quantize=True, out=out)
        tp.tp_rmsnorm_backward(dY, out["S"], w, out["rstd"], out=back, ws=ws)
    for seed in (30, 31):
        X.copy_(rows(T, h, torch.bfloat16, seed))
        graph.replay()
        ref = tp.tp_rmsnorm_forward(X, w, R, quantize=True)
        refb = tp.tp_rmsnorm_backward(dY, ref["S"], w, ref["rstd"])
        for k, v in {**ref, **refb}.items():
            mine = {**out, **back}[k]
            assert torch.equal(mine.view(torch.uint8), v.view(torch.uint8)), k


def test_rows_that_two_blocks_share_in_a_graph():
    gpu_or_skip()
    T, h = 200, 8208
    S, dY, w = rows(T, h, torch.bfloat16, 16), rows(T, h, torch.bfloat16, 18), weight(h)
    rstd = norm_forward(S, w, EPS)[1].float()
    out = tp.tp_rmsnorm_backward(dY, S, w, rstd)
    ws = torch.empty(tp.rmsnorm_workspace_bytes(T, h), dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for _ in range(3):
            tp.tp_rmsnorm_backward(dY, S, w, rstd, out=out, ws=ws)
    for seed in (30, 31):
        dY.copy_(rows(T, h, torch.bfloat16, seed))
        graph.replay()
        ref = tp.tp_rmsnorm_backward(dY, S, w, rstd)
        assert torch.equal(out["dX"], ref["dX"]) and torch.equal(out["dw"], ref["dw"])


def test_an_output_that_does_not_fit_is_torchs_own_error():
    # copies of 512 GiB, more than the device has: torch's error, which a program may catch and go on
    gpu_or_skip()
    ids = torch.zeros(1 << 20, 32, dtype=torch.int32, device="cuda")
    plan = {"row": ids, "offsets": torch.zeros(2, dtype=torch.int32, device="cuda")}
    big = torch.zeros(1 << 20, 8192, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(torch.OutOfMemoryError):
        tp.tp_expert_dispatch_forward(big, plan)
    assert tp.tp_rmsnorm_forward(big[:2], weight(8192))["Y"].shape == (2, 8192)
