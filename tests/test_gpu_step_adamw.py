"""The AdamW step against the plain 64-bit form and against elementary 32-bit
operations (the same bits): every mix of parameter, master, gradient and state
types, lengths of one, around a group and a block of work, lists longer than a
launch holds, gradients that are not finite, tensors of more than 2^31 values,
another stream, a captured step with device scalars.

Bounds (_step_ref): m is two products and a sum of values with up to 4
roundings each, v has up to 6; the update divides by a root, with 16 roundings
at most altogether; the parameter adds 4. Constants are rounded to fp32 once
each.
"""

import math

import pytest
import torch

import vocab_ce_gb300 as tp
from _parity import gpu_or_skip
from _step_ref import D, E32, GROUP, U, adamw, codes_near, groups, near, spread

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
HYPER = dict(lr=2e-3, beta1=0.9, beta2=0.95, eps=1e-8, step=7, grad_scale=0.5)
LENGTHS = [1, 7, 8, 9, 127, 128, 129, 255, 2047, 2048, 2049, 5000, 40_000]
KINDS = [(F32, F32, False), (F32, BF, False), (BF, BF, False), (BF, F32, False), (BF, BF, True), (BF, F32, True)]


def normal(n, seed, std=1.0):
    return std * torch.randn(n, generator=torch.Generator(device="cuda").manual_seed(seed), device="cuda")


def quantize(x):
    """Codes and scales of the library's 8-bit format, in elementary 32-bit operations."""
    b = groups(x)
    a = torch.where(b.isfinite(), b.abs(), 0.0)
    scale = (a.amax(-1) * (1.0 / 448.0)).clamp_min(2.0 ** -126)
    t = torch.where(b.isfinite(), b * scale.reciprocal()[:, None], float("nan"))
    return t.to(torch.float8_e4m3fn).reshape(-1)[:x.numel()], scale


def tensors(n, p_dtype, g_dtype, master, bits, seed):
    p32 = normal(n, seed, 0.05)
    st = {"m": normal(n, seed + 1, 1e-3), "v": normal(n, seed + 2, 1e-3).square()}
    if bits == 8:
        (mq, ms), (rq, rs) = quantize(st["m"]), quantize(st["v"].sqrt())
        st = {"m_q": mq, "m_scale": ms, "r_q": rq, "r_scale": rs}
    return dict(p=p32.to(p_dtype, copy=True), master=p32.clone() if master else None,
                g=normal(n, seed + 3, 2e-3).to(g_dtype), st=st)


def copy(t):
    return dict(p=t["p"].clone(), master=None if t["master"] is None else t["master"].clone(), g=t["g"],
                st={k: v.clone() for k, v in t["st"].items()})


def step(ts, wd=0.1, **more):
    h = {**HYPER, **more}
    tp.adamw_step([t["p"] for t in ts], [t["g"] for t in ts], [t["st"] for t in ts],
                  masters=[t["master"] for t in ts], weight_decay=wd, **h)


def bits_of(t):
    return [x.contiguous().view(torch.uint8) for x in (t["p"], t["master"], *t["st"].values()) if x is not None]


def same(a, b, what=""):
    for x, y in zip(bits_of(a), bits_of(b)):
        assert torch.equal(x, y), what


def elementary(t, wd):
    """One step in separate 32-bit operations, in place."""
    h, st, n = HYPER, t["st"], t["p"].numel()
    g = t["g"].float() * h["grad_scale"]
    if "m" in st:
        m, v = st["m"], st["v"]
    else:
        m = (groups(st["m_q"].float()) * st["m_scale"][:, None]).reshape(-1)[:n]
        v = (groups(st["r_q"].float()) * st["r_scale"][:, None]).reshape(-1)[:n]
        v = v * v
    m = m * h["beta1"] + g * (1.0 - h["beta1"])
    v = v * h["beta2"] + (g * g) * (1.0 - h["beta2"])
    r = v.sqrt()
    p = (t["p"] if t["master"] is None else t["master"]).float()
    bc1, bc2 = 1.0 - h["beta1"] ** h["step"], 1.0 - h["beta2"] ** h["step"]
    p = p * (1.0 - h["lr"] * wd) - (m / (r * (1.0 / math.sqrt(bc2)) + h["eps"])) * (h["lr"] / bc1)
    if t["master"] is not None:
        t["master"].copy_(p)
    t["p"].copy_(p)
    if "m" in st:
        st["m"].copy_(m)
        st["v"].copy_(v)
    else:
        for name, x in (("m", m), ("r", r)):
            q, s = quantize(x)
            st[name + "_q"].copy_(q)
            st[name + "_scale"].copy_(s)


def check64(old, new, wd, what):
    h, n = HYPER, old["p"].numel()
    if "m" in old["st"]:
        m0, v0 = old["st"]["m"].to(D), old["st"]["v"].to(D)
    else:
        m0 = old["st"]["m_q"].float().to(D) * spread(old["st"]["m_scale"], n)
        v0 = (old["st"]["r_q"].float().to(D) * spread(old["st"]["r_scale"], n)).pow(2)
    p0 = (old["p"] if old["master"] is None else old["master"]).to(D)
    g = old["g"].to(D)
    p, m, v, u = adamw(p0, g, m0, v0, h["lr"], h["step"], h["beta1"], h["beta2"], h["eps"], wd, h["grad_scale"])
    em = 4 * E32 * (h["beta1"] * m0.abs() + (1 - h["beta1"]) * (g * h["grad_scale"]).abs()) + 2.0 ** -149
    ev = 6 * E32 * v + 2.0 ** -148
    # m's terms can cancel: its error reaches the update through |lr / denominator|
    per_m = h["lr"] / (1 - h["beta1"] ** h["step"]) / ((v / (1 - h["beta2"] ** h["step"])).sqrt() + h["eps"])
    ep = 16 * E32 * u + per_m * em + 4 * E32 * p0.abs()
    got = (new["p"] if new["master"] is None else new["master"])
    near(got, p, ep + (U[got.dtype] * p.abs() if got.dtype == BF else 0.0), what + " p")
    if new["master"] is not None:
        assert torch.equal(new["p"], new["master"].to(BF)), what
    if "m" in new["st"]:
        near(new["st"]["m"], m, em, what + " m")
        near(new["st"]["v"], v, ev, what + " v")
    else:
        codes_near(new["st"]["m_q"], new["st"]["m_scale"], m, em, what + " m")
        codes_near(new["st"]["r_q"], new["st"]["r_scale"], v.sqrt(), 8 * E32 * v.sqrt() + 2.0 ** -140, what + " r")


@pytest.mark.parametrize("bits", [8, 32])
@pytest.mark.parametrize("p_dtype,g_dtype,master", KINDS)
def test_step(p_dtype, g_dtype, master, bits):
    gpu_or_skip()
    old = [tensors(n, p_dtype, g_dtype, master, bits, 10 * i) for i, n in enumerate(LENGTHS)]
    new, plain = [copy(t) for t in old], [copy(t) for t in old]
    wd = [0.1 * (i % 2) for i in range(len(old))]
    step(new, wd)
    for n, o, t, q, d in zip(LENGTHS, old, new, plain, wd):
        check64(o, t, d, f"n={n}")
        elementary(q, d)
        same(t, q, f"n={n}")


def test_a_list_gives_what_its_tensors_give_alone():
    # mixed kinds in one list, and more tensors than one launch holds
    gpu_or_skip()
    kinds = [(k, b) for k in KINDS for b in (8, 32)]
    for count in (13, 48, 49, 400, 401, 830):
        many = [tensors(1 + (97 * i) % 700, *kinds[i % 12][0], kinds[i % 12][1], i) for i in range(count)]
        alone = [copy(t) for t in many[:: max(1, count // 20)]]
        step(many)
        for t in alone:
            step([t])
        for t, a in zip(many[:: max(1, count // 20)], alone):
            same(t, a, str(count))


def test_first_step_from_zero_state_and_steps_without_a_gradient():
    gpu_or_skip()
    for bits in (8, 32):
        p = normal(300, 1)
        st, g = tp.adamw_state(p, bits), normal(300, 2)
        q = p.clone()
        tp.adamw_step([q], [g], [st], lr=1e-2, step=1, eps=0.0, weight_decay=0.0)
        # the first step moves every value by lr against its gradient's sign
        near(q, p.to(D) - 1e-2 * g.to(D).sign(), 16 * E32 * 1e-2 + 4 * E32 * p.to(D).abs(), f"{bits}")
        tp.adamw_step([q], [torch.zeros_like(g)], [st], lr=1e-2, step=2)
        assert bool(q.isfinite().all())
    st = tp.adamw_state(p, 8)
    q = p.clone()
    tp.adamw_step([q], [torch.zeros_like(p)], [st], lr=1e-2, step=1)
    assert torch.equal(q, p) and not st["m_q"].float().any() and bool((st["r_scale"] == 2.0 ** -126).all())


def test_gradients_that_are_not_finite_stay_in_their_places():
    gpu_or_skip()
    for bits in (8, 32):
        t = tensors(1000, F32, F32, False, bits, 3)
        t["g"][5], t["g"][200], t["g"][999] = float("inf"), float("nan"), -float("inf")
        clean = copy(t)
        clean["g"] = t["g"].clone()
        clean["g"][5] = clean["g"][200] = clean["g"][999] = 0.0
        step([t])
        step([clean])
        hit = torch.zeros(1000, dtype=torch.bool, device="cuda")
        hit[5] = hit[200] = hit[999] = True
        assert bool(t["p"][hit].isnan().all()) and torch.equal(t["p"][~hit], clean["p"][~hit])
        if bits == 32:
            assert bool((~t["st"]["m"][hit].isfinite()).all())
            assert torch.equal(t["st"]["m"][~hit], clean["st"]["m"][~hit])
        else:
            for key in ("m_q", "r_q"):
                q = t["st"][key].float()
                assert bool(q[hit].isnan().all()) and bool(q[~hit].isfinite().all())
            assert bool(t["st"]["m_scale"].isfinite().all()) and bool(t["st"]["r_scale"].isfinite().all())


def test_tiny_and_huge_groups():
    # groups whose squares are near the bottom and the top of fp32
    gpu_or_skip()
    n = 3 * GROUP
    t = tensors(n, F32, F32, False, 8, 4)
    t["g"][:GROUP] = 1e-15
    t["g"][GROUP:2 * GROUP] = 1e18
    for key in t["st"]:
        t["st"][key].view(torch.uint8).zero_()
    old, plain = copy(t), copy(t)
    step([t])
    elementary(plain, 0.1)
    same(t, plain)
    assert bool(t["p"].isfinite().all()) and bool(t["st"]["m_scale"].isfinite().all())
    check64(old, t, 0.1, "tiny and huge")


def test_many_values():
    gpu_or_skip()
    n, at = 2 ** 31 + 2 * 2048 + 5, 2 ** 31 - 2048
    p = torch.zeros(n, dtype=BF, device="cuda")
    g = torch.zeros(n, dtype=BF, device="cuda")
    st = tp.adamw_state(p, 8)
    g[at:] = normal(n - at, 5).to(BF)
    p[at:] = normal(n - at, 6).to(BF)
    q, h = p[at:].clone(), g[at:].clone()
    qs = tp.adamw_state(q, 8)
    tp.adamw_step([p], [g], [st], **HYPER)
    tp.adamw_step([q], [h], [qs], **HYPER)
    assert torch.equal(p[at:], q) and not p[:10_000].any()
    assert torch.equal(st["m_q"][at:].view(torch.uint8), qs["m_q"].view(torch.uint8))
    assert torch.equal(st["r_scale"][at // GROUP:], qs["r_scale"])


def test_refused_arguments():
    gpu_or_skip()
    p, g = normal(64, 1), normal(64, 2)
    st = tp.adamw_state(p)
    before = p.clone()
    ok = dict(lr=1e-3, step=1)
    with pytest.raises(ValueError, match="twice"):
        tp.adamw_step([p, p], [g, g], [st, tp.adamw_state(p)], **ok)
    with pytest.raises(ValueError, match="shape"):
        tp.adamw_step([p], [g[:32]], [st], **ok)
    with pytest.raises(ValueError, match="contiguous"):
        tp.adamw_step([normal(128, 1)[::2]], [g], [st], **ok)
    with pytest.raises(ValueError, match="float16"):
        tp.adamw_step([p], [g.half()], [st], **ok)
    with pytest.raises(ValueError, match="states"):
        tp.adamw_step([p], [g], [], **ok)
    with pytest.raises(ValueError, match="weight_decay"):
        tp.adamw_step([p], [g], [st], weight_decay=[0.1, 0.2], **ok)
    with pytest.raises(ValueError, match="scalars"):
        tp.adamw_step([p], [g], [st], scalars=torch.zeros(3, device="cuda"), **ok)
    with pytest.raises(tp.TpceError):
        tp.adamw_step([p], [g], [st], lr=1e-3, step=0)
    with pytest.raises(tp.TpceError):                       # a start that is not on 16 bytes
        tp.adamw_step([normal(65, 1)[1:]], [g], [st], **ok)
    assert torch.equal(p, before)
    empty = torch.empty(0, device="cuda")
    tp.adamw_step([empty, p], [empty, g], [tp.adamw_state(empty, 8), st], **ok)
    assert not torch.equal(p, before)
    tp.adamw_step([], [], [], **ok)


def test_on_another_stream():
    gpu_or_skip()
    a = [tensors(n, BF, BF, True, 8, n) for n in (3000, 77)]
    b = [copy(t) for t in a]
    step(a)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    step(b, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    for x, y in zip(a, b):
        same(x, y)


def test_captured_step_reads_its_scalars():
    gpu_or_skip()
    a = [tensors(n, k[0], k[1], k[2], bits, n) for n, k, bits in ((3000, KINDS[4], 8), (500, KINDS[0], 32))]
    b = [copy(t) for t in a]
    scalars = tp.adamw_scalars(1e-3, 1).cuda()
    for t in a:
        t["g"] = t["g"].clone()
    warm = [copy(t) for t in a]
    step(warm, scalars=scalars)                              # loads the kernel
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(a, scalars=scalars)
    for i in (1, 2, 3):
        h = dict(lr=1e-3 * i, step=i, grad_scale=1.0 / i)
        for x, y in zip(a, b):
            x["g"].copy_(normal(x["g"].numel(), 50 + i, 1e-2))
            y["g"] = x["g"]
        scalars.copy_(tp.adamw_scalars(h["lr"], h["step"], HYPER["beta1"], HYPER["beta2"], h["grad_scale"]))
        graph.replay()
        step(b, **h)
        for x, y in zip(a, b):
            # 1 - lr wd is rounded on the device here and in 64 bits there: one step of it
            px, py = (t["p"] if t["master"] is None else t["master"] for t in (x, y))
            near(px, py, 8 * i * E32 * py.to(D).abs(), f"step {i}")
            for key in x["st"]:
                assert torch.equal(x["st"][key].view(torch.uint8), y["st"][key].view(torch.uint8)), key
