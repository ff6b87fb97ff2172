"""What the training-step calls write in place counts as changed for autograd: a
backward pass that has saved the old values is refused by torch, instead of
giving wrong gradients."""

import pytest
import torch

import vocab_ce_gb300 as tp
from _parity import gpu_or_skip

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


def normal(shape, seed, dtype=F32):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(shape, generator=g, device="cuda").to(dtype)


def versions(xs):
    return [x._version for x in xs]


@pytest.mark.parametrize("bits", [8, 32])
def test_a_step_between_forward_and_backward_is_seen(bits):
    gpu_or_skip()
    p, x = normal(300, 1).requires_grad_(), normal(300, 2).requires_grad_()
    loss = (p * x).sum()
    tp.adamw_step([p.detach()], [normal(300, 3)], [tp.adamw_state(p, bits)], lr=0.1, step=1)
    with pytest.raises(RuntimeError, match="inplace"):
        loss.backward()


def test_a_step_changes_parameters_and_masters():
    gpu_or_skip()
    w, master, g = normal(300, 1, BF), normal(300, 2), normal(300, 3)
    p = normal(40, 4)
    states = [tp.adamw_state(w, 8), tp.adamw_state(p, 32)]
    written = [w, master, p]
    before, other = versions(written), g._version
    args = ([w, p], [g, normal(40, 5)], states)
    tp.adamw_step(*args, lr=0.1, step=1, masters=[master, None])
    assert versions(written) == [v + 1 for v in before] and g._version == other
    with pytest.raises(tp.TpceError):
        tp.adamw_step(*args, lr=0.1, step=0, masters=[master, None])   # refused: nothing is written
    assert versions(written) == [v + 1 for v in before]


def test_outputs_given_by_the_caller():
    gpu_or_skip()
    T, h, k, E = 5, 64, 2, 4
    X, R, w = normal((T, h), 1, BF), normal((T, h), 2, BF), normal(h, 3)
    new = tp.tp_rmsnorm_forward(X, w, R=R, quantize=True)
    out = {n: torch.empty_like(x) for n, x in new.items()}
    out["S"] = R
    tp.tp_rmsnorm_forward(X, w, R=R, quantize=True, out=out)
    assert versions(out.values()) == [1] * 5 and versions([X, w]) == [0, 0]
    dY = normal((T, h), 4, BF)
    res = tp.tp_rmsnorm_backward(dY, new["S"], w, new["rstd"], out={"dX": dY})
    assert res["dX"] is dY and versions([dY, new["S"], new["rstd"], res["dw"]]) == [1, 0, 0, 0]
    ids = torch.randint(0, E, (T, k), device="cuda", dtype=torch.int32)
    plan = tp.tp_expert_plan(ids, E)
    again = tp.tp_expert_plan(ids, E, out=plan)
    assert versions(again.values()) == [1] * 3
    Xs, Z, dX = torch.empty(T * k, h, dtype=BF, device="cuda"), torch.empty_like(X), torch.empty_like(X)
    weights = torch.rand(T, k, device="cuda")
    tp.tp_expert_dispatch_forward(X, plan, out=Xs)
    tp.tp_expert_combine_forward(Xs, plan, weights, out=Z)
    tp.tp_expert_dispatch_backward(Xs, plan, out=dX)
    grads = {"dYs": torch.empty_like(Xs), "dweights": torch.empty_like(weights)}
    tp.tp_expert_combine_backward(Z, Xs, plan, weights, out=grads)
    assert versions([Xs, Z, dX, *grads.values()]) == [1] * 5 and versions([weights, ids]) == [0, 0]


def test_tensors_of_inference_mode():
    gpu_or_skip()
    with torch.inference_mode():
        p, g = normal(100, 1), normal(100, 2)
        st = tp.adamw_state(p)
    before = p.clone()
    tp.adamw_step([p], [g], [st], lr=0.1, step=1)                      # outside the mode
    with torch.inference_mode():
        tp.adamw_step([p], [g], [st], lr=0.1, step=2)
        assert not torch.equal(p, before)
