"""AdamW with 8-bit states over many steps, beside the same run with 32-bit
states: how large a step may become, and how far a root may lag."""

import math

import pytest
import torch

import vocab_ce_gb300 as tp
from _parity import gpu_or_skip

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
LEAST = 2.0 ** -9   # the smallest code


def generator(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def largest_step(bits, size, decades, steps=400, groups=500):
    """In units of lr: gradients present one step in twenty, their sizes spread inside every group."""
    g, n = generator(0), groups * 128
    sizes = size * 10.0 ** (-decades * torch.rand(n, generator=g, device="cuda"))
    p = torch.zeros(n, device="cuda")
    st, most = tp.adamw_state(p, bits), torch.zeros((), device="cuda")
    for t in range(1, steps + 1):
        there = torch.rand(n, generator=g, device="cuda") < 0.05
        grad = torch.where(there, sizes * torch.randn(n, generator=g, device="cuda"), 0.0)
        p.zero_()
        tp.adamw_step([p], [grad], [st], lr=1.0, step=t)
        most = torch.maximum(most, p.abs().max())
    return float(most)


@pytest.mark.parametrize("decades", [3, 5])
@pytest.mark.parametrize("size", [1e-3, 1.0, 10.0])
def test_rare_gradients_make_no_huge_steps(size, decades):
    """AdamW does not see the gradients' size. A moment that no longer has a gradient stops shrinking at codes of up to
    4.5 smallest ones (0.9 of them rounds to themselves) and its root is at least one: the step is then up to 4.5 times
    the ratio of the group's largest moment and root, which 32-bit states bound."""
    gpu_or_skip()
    assert largest_step(8, size, decades) <= 5.0 * largest_step(32, size, decades)


@pytest.mark.parametrize("p_dtype,master", [(F32, False), (BF, False), (BF, True)])
@pytest.mark.parametrize("n", [1, 128, 300, 2048 + 5])
def test_a_root_that_is_not_zero_keeps_a_code(n, p_dtype, master):
    gpu_or_skip()
    p32 = torch.randn(n, generator=generator(1), device="cuda")
    grad = torch.zeros(n, device="cuda")
    grad[0::128] = 1.0                       # each group's largest
    grad[1::128], grad[2::128], grad[5::128] = 1e-7, -1e-12, float("nan")
    p, st = p32.to(p_dtype), tp.adamw_state(p32, 8)
    tp.adamw_step([p], [grad], [st], lr=1e-3, step=1, masters=[p32.clone()] if master else None)
    r, nan = st["r_q"].float(), grad.isnan()
    assert torch.equal(r.isnan(), nan)
    assert bool((r[0::128] == 448.0).all())
    small = (grad != 0) & ~nan
    small[0::128] = False
    assert bool((r[small] == LEAST).all())   # 1e-7 / 1 and 1e-12 / 1 of 448, below half the smallest code
    assert bool((r[grad == 0] == 0.0).all())
    # a group of zeros, and one whose values are all alike
    st, zero = tp.adamw_state(p32, 8), torch.zeros(n, device="cuda")
    tp.adamw_step([p], [zero], [st], lr=1e-3, step=1)
    assert not st["r_q"].float().any()
    tp.adamw_step([p], [zero + 1e-15], [st], lr=1e-3, step=2)
    assert bool((st["r_q"].float() == 448.0).all()) and math.isclose(float(st["r_scale"][0]) * 448.0,
                                                                     1e-15 * math.sqrt(1 - 0.999), rel_tol=1e-5)


# ------------------------------------------------------------------ how far a root may lag
def roots(st):
    """A state's roots, and their scales spread over the values."""
    if "v" in st:
        return st["v"].sqrt(), None
    n = st["r_q"].numel()
    s = st["r_scale"].repeat_interleave(128)[:n]
    return st["r_q"].float() * s, s


def lag(beta2):
    """Rounded to nearest, a root that stays has (17/16 r)^2 >= beta2 r^2 + (1 - beta2) g^2: half a step of a code is
    at most 1/16 of it. So r >= g times this."""
    return math.sqrt((1.0 - beta2) / ((17.0 / 16.0) ** 2 - beta2))


@pytest.mark.parametrize("beta2", [0.95, 0.99, 0.999])
@pytest.mark.parametrize("p_dtype,master", [(F32, False), (BF, True)])
def test_rounded_to_nearest_a_root_lags_no_further_than_stated(beta2, p_dtype, master):
    gpu_or_skip()
    n, steps = 100 * 128, 3000
    size = 10.0 ** (-2.0 - torch.rand(n, generator=generator(1), device="cuda"))
    size[0::128] = 1.0
    sign = torch.where(torch.rand(n, generator=generator(2), device="cuda") < 0.5, 1.0, -1.0)
    p32 = torch.zeros(n, device="cuda")
    p, held = (p32.to(p_dtype), p32) if master else (p32, None)
    st = tp.adamw_state(p, 8)
    for t in range(1, 2 * steps + 1):
        if t == steps + 1:
            size[size < 0.5] *= 20.0    # still below the largest
        p.zero_()
        p32.zero_()
        tp.adamw_step([p], [sign * size], [st], lr=1.0, step=t, beta2=beta2, masters=[held])
    r, _ = roots(st)
    assert bool((r >= 0.99 * lag(beta2) * size).all()), float((r / size).min())
    # the steps: of 1 lr with roots that are right; the moment is off by at most 1/16 of nine tenths of itself
    assert float(p32.abs().max()) <= 1.07 / lag(beta2)


def run_noise(bits, rounding, beta2, steps=3000, groups=100):
    """Normal gradients whose size grows by 5 halfway, but for each group's largest; the state and the last step."""
    g, n = generator(3), groups * 128
    size = 10.0 ** (-1.0 - torch.rand(n, generator=g, device="cuda"))
    size[0::128] = 1.0
    p = torch.zeros(n, device="cuda")
    st = tp.adamw_state(p, bits)
    for t in range(1, 2 * steps + 1):
        if t == steps + 1:
            size = torch.where(size < 0.5, 5.0 * size, size)
        p.zero_()
        tp.adamw_step([p], [size * torch.randn(n, generator=g, device="cuda")], [st], lr=1.0, step=t, beta2=beta2,
                      rounding=rounding)
    return roots(st)[0], p


@pytest.mark.parametrize("beta2", [0.95, 0.99, 0.999])
def test_rounded_at_random_roots_and_steps_follow_the_gradients(beta2):
    """The expectation of a root is the exact one's, so its median stays near it (simulated on the CPU beforehand: 0.98
    to 1.00, and 0.38 rounded to nearest with beta2 = 0.999); an update divides by it."""
    gpu_or_skip()
    want, step = run_noise(32, "nearest", beta2)
    r, moved = run_noise(8, "random", beta2)
    assert 0.9 <= float((r / want).median()) <= 1.1
    ratio = (moved / step)[step.abs() > 1e-2]
    assert 0.85 <= float(ratio.median()) <= 1.2


def run_ended(bits, rounding, beta1, steps=400, after=1000, groups=100):
    """How far parameters move whose gradients end, beside others whose stay, in a group with a steady largest one."""
    g, n = generator(4), groups * 128
    size = 10.0 ** (-1.0 - torch.rand(n, generator=g, device="cuda"))
    ended = torch.arange(n, device="cuda") % 128 >= 64
    p, st = torch.zeros(n, device="cuda"), tp.adamw_state(torch.zeros(n, device="cuda"), bits)
    for t in range(1, steps + after + 1):
        grad = size * torch.randn(n, generator=g, device="cuda")
        grad[0::128] = 3.0
        if t > steps:
            grad[ended] = 0.0
        if t == steps + 1:
            p.zero_()
        tp.adamw_step([p], [grad], [st], lr=1.0, step=t, beta1=beta1, rounding=rounding)
    return p[ended].abs()


@pytest.mark.parametrize("beta1", [0.9, 0.95, 0.99])
def test_rounded_at_random_a_parameter_without_gradients_comes_to_rest(beta1):
    """Simulated on the CPU beforehand: medians within 6% of the 32-bit run's, the largest 1.6 times; rounded to
    nearest, a moment that stays moves it on (35 times the 32-bit run's at 0.95)."""
    gpu_or_skip()
    want, got = run_ended(32, "nearest", beta1), run_ended(8, "random", beta1)
    assert 0.8 <= float(got.median() / want.median()) <= 1.25
    assert float(got.max()) <= 3.0 * float(want.max())


# ------------------------------------------------------------------ random rounding, one step
def state8(n, seed, spread=3.0):
    """Codes and scales as steps leave them: the largest of a group at code 448."""
    from test_gpu_step_adamw import quantize
    size = 10.0 ** (-spread * torch.rand(n, generator=generator(seed), device="cuda"))
    m = 1e-3 * size * torch.randn(n, generator=generator(seed + 1), device="cuda")
    r = 1e-3 * size * (0.5 + torch.rand(n, generator=generator(seed + 2), device="cuda"))
    (mq, ms), (rq, rs) = quantize(m), quantize(r)
    g = 1e-3 * size * torch.randn(n, generator=generator(seed + 3), device="cuda")
    return {"m_q": mq, "m_scale": ms, "r_q": rq, "r_scale": rs}, g


def copy(st):
    return {k: v.clone() for k, v in st.items()}


def same(a, b):
    return all(torch.equal(a[k].view(torch.uint8), b[k].view(torch.uint8)) for k in a)


def between(t):
    """The distance of the two codes around t (in units of the scale)."""
    return torch.exp2(t.log2().floor().clamp_min(-6.0) - 3.0)


def check_neighbours(q, t, inside, what):
    """Codes q of exact values t >= 0: each a neighbour, and right on average wherever between the codes t lies. A
    choice is off by less than a step with mean 0, so the mean of N is within 5 half steps / sqrt(N) of 0."""
    off = (q - t) / between(t)
    assert bool((off[inside].abs() < 1.0 + 1e-5).all()), what
    for lo, hi in ((0.0, 1.0), (0.0, 0.25), (0.25, 0.5), (0.5, 0.75), (0.75, 1.0)):
        f = (t / between(t)).frac()
        part = inside & (f >= lo) & (f < hi)
        count = int(part.sum())                        # (a step of beta2 = 0.999 moves few roots far)
        assert count == 0 or abs(float(off[part].mean())) <= 5.0 * 0.5 / math.sqrt(count), (what, lo)


@pytest.mark.parametrize("spread", [0.0, 3.0, 5.0])
def test_a_random_code_is_a_neighbour_and_right_on_average(spread):
    gpu_or_skip()
    n = 1 << 20
    st, g = state8(n, 10, spread)
    m = st["m_q"].float() * st["m_scale"].repeat_interleave(128)
    r = st["r_q"].float() * st["r_scale"].repeat_interleave(128)
    exact = {"m": m, "v": r * r}                       # the same step with its state left in 32 bits
    near, rand = copy(st), copy(st)
    p = [torch.zeros(n, device="cuda") for _ in range(3)]
    for x, s, how in zip(p, (exact, near, rand), ("nearest", "nearest", "random")):
        tp.adamw_step([x], [g], [s], lr=1e-3, step=5, rounding=how)
    # nothing but the codes differs
    assert torch.equal(p[0], p[1]) and torch.equal(p[0], p[2])
    assert all(torch.equal(near[k], rand[k]) for k in ("m_scale", "r_scale"))
    t = exact["v"].double().sqrt() / rand["r_scale"].double().repeat_interleave(128)
    q = rand["r_q"].double()
    check_neighbours(q, t, (t > LEAST) & (t < 447.0), "root")   # below: the smallest code; above: the largest
    assert bool((q[t <= LEAST] == LEAST).all()) and bool((q[t >= 447.0] >= 416.0).all())
    signed = exact["m"].double() / rand["m_scale"].double().repeat_interleave(128)
    t, q = signed.abs(), rand["m_q"].double()
    assert bool((q * signed >= 0).all())               # the sign stays, or the value is zero
    check_neighbours(q.abs(), t, (t > 0) & (t < 447.0), "moment")


def test_random_rounding_repeats_itself_and_varies_with_the_step():
    gpu_or_skip()
    sizes = [5, 128, 700, 2053, 300, 4096]
    made = [state8(n, 20 + i) for i, n in enumerate(sizes)]

    def run(which, step=9, rounding="random"):
        sts = [copy(made[i][0]) for i in which]
        ps = [torch.zeros(sizes[i], device="cuda") for i in which]
        tp.adamw_step(ps, [made[i][1] for i in which], sts, lr=1e-3, step=step, rounding=rounding)
        return sts

    whole = run(range(6))
    assert all(same(a, b) for a, b in zip(whole, run(range(6))))
    for i in range(6):
        assert same(whole[i], run([i])[0])             # alone, and wherever it is in the list
    assert same(whole[5], run([5, 2])[0])
    other = run(range(6), step=10)
    # where a value lies at f between two codes, two independent choices differ with 2 f (1 - f)
    differ, chance = 0, 0.0
    for (st, g), a, b in zip(made, whole, other):
        n = g.numel()
        r = st["r_q"].float() * st["r_scale"].repeat_interleave(128)[:n]
        exact = {"m": torch.zeros(n, device="cuda"), "v": r * r}
        tp.adamw_step([torch.zeros(n, device="cuda")], [g], [exact], lr=1e-3, step=9)
        t = exact["v"].double().sqrt() / a["r_scale"].double().repeat_interleave(128)[:n]
        f = (t / torch.exp2(t.log2().floor().clamp_min(-6.0) - 3.0)).frac()
        chance += float((2.0 * f * (1.0 - f)).sum())
        differ += int((a["r_q"].float() != b["r_q"].float()).sum())
    assert chance > 50 and abs(differ - chance) <= 5.0 * math.sqrt(chance), (differ, chance)
    assert any(not same(a, b) for a, b in zip(whole, run(range(6), rounding="nearest")))


def test_random_rounding_leaves_zeros_nans_and_32_bits_alone():
    gpu_or_skip()
    n = 700
    g = torch.randn(n, generator=generator(5), device="cuda")
    g[3], g[200], g[500], g[128:136] = float("nan"), float("inf"), 1e-15, 0.0
    states = [tp.adamw_state(g, 8), tp.adamw_state(g, 32)]
    alone = tp.adamw_state(g, 32)
    p = [torch.zeros(n, device="cuda") for _ in range(3)]
    tp.adamw_step(p[:2], [g, g], states, lr=1e-3, step=1, rounding="random")
    tp.adamw_step(p[2:], [g], [alone], lr=1e-3, step=1)
    r, odd = states[0]["r_q"].float(), ~g.isfinite()
    assert torch.equal(r.isnan(), odd) and bool((r[g == 0] == 0).all()) and float(r[500]) == LEAST
    assert bool((r[~odd & (g != 0)] >= LEAST).all()) and bool(states[0]["r_scale"].isfinite().all())
    m = states[0]["m_q"].float()
    assert torch.equal(m.isnan(), odd) and bool((m[g == 0] == 0).all()) and bool(states[0]["m_scale"].isfinite().all())
    assert same(states[1], alone) and torch.equal(p[1][~odd], p[2][~odd])


def test_random_rounding_in_a_captured_step():
    gpu_or_skip()
    st, g = state8(3000, 30)
    eager, captured = copy(st), copy(st)
    p = [torch.zeros(3000, device="cuda") for _ in range(3)]
    scalars = tp.adamw_scalars(1e-3, 6).cuda()
    tp.adamw_step([p[0]], [g], [copy(st)], lr=1e-3, step=6, scalars=scalars, rounding="random")   # loads the kernel
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        tp.adamw_step([p[1]], [g], [captured], lr=1e-3, step=6, scalars=scalars, rounding="random")
    graph.replay()
    tp.adamw_step([p[2]], [g], [eager], lr=1e-3, step=6, rounding="random")
    assert same(eager, captured)
    for k, v in st.items():
        captured[k].copy_(v)
    scalars.copy_(tp.adamw_scalars(1e-3, 7))
    graph.replay()                                     # another step's numbers: other codes
    assert not same({"r_q": eager["r_q"]}, {"r_q": captured["r_q"]})


def test_one_list_may_round_either_way():
    # by the C ABI, where it is each tensor's: in the same launch, tensors rounded to nearest and with 32-bit states
    # keep their bits
    gpu_or_skip()
    from vocab_ce_gb300._lib import AdamwTensor, lib
    sizes = [(700, "nearest"), (5000, "random"), (300, None), (129, "random"), (2049, "nearest")]
    made = [state8(n, 40 + i) for i, (n, _) in enumerate(sizes)]

    def fresh():
        return [(torch.zeros(n, device="cuda"), g, copy(st) if how else tp.adamw_state(g, 32))
                for (n, how), (st, g) in zip(sizes, made)]

    one, alone = fresh(), fresh()
    table = (AdamwTensor * len(sizes))()
    for e, (p, g, st), (n, how) in zip(table, one, sizes):
        e.p, e.g, e.n, e.p_dtype, e.g_dtype = p.data_ptr(), g.data_ptr(), n, 1, 1
        e.state_bits = 32 if how is None else 8 | (256 if how == "random" else 0)
        names = ("m", "v") if how is None else ("m_q", "r_q", "m_scale", "r_scale")
        for field, name in zip(("m", "v", "m_scale", "v_scale"), names):
            setattr(e, field, st[name].data_ptr())
    stream = torch.cuda.current_stream().cuda_stream
    assert lib().tp_adamw_step(table, len(sizes), 1e-3, 0.9, 0.999, 1e-8, 5, 1.0, None, stream) == 0
    for (p, g, st), (q, h, su), (_, how) in zip(one, alone, sizes):
        tp.adamw_step([q], [h], [su], lr=1e-3, step=5, rounding=how or "nearest")
        assert torch.equal(p, q) and same(st, su), how
