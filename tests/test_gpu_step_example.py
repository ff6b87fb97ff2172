"""The training-step operators together: examples/expert_layer.py's gradients
against autograd in 64 bits on the same weights and choices, its training run,
and chains of calls that nothing waits between.

Gradients: a path rounds at most 12 intermediates to bf16 on the way from the
inputs to a weight's gradient (Y, the router's or the experts' activations, Ys,
Z, S, H, dl, dH, dS, dYs, dU, dXs and their sum), each off by at most 2^-8 and
2^-8 / sqrt(3) root mean square of its values; independent ones add in squares:
sqrt(13) 2^-8 / sqrt(3) = 0.8% of the gradient's norm where no sum cancels. The
loss's gradient cancels (softmax minus one-hot, and the norms' projections):
three times that is allowed, 2.5% in the 2-norm.
"""

import os
import sys

import pytest
import torch

import vocab_ce_gb300 as tp
from _parity import gpu_or_skip
from _step_ref import D

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))

pytestmark = pytest.mark.gpu


def reference(layer, S, targets, ids, eps=1e-6):
    """The layer in 64 bits by autograd, on the same weights and the same choices."""
    p = {n: x.to(D).requires_grad_(True) for n, x in layer.params.items()}
    x = S.to(D)

    def norm(s, w):
        return s * (s.pow(2).mean(-1, keepdim=True) + eps).rsqrt() * w
    Y = norm(x, p["w1"])
    weights = (Y @ p["router"]).gather(1, ids).softmax(-1)
    Z = torch.zeros_like(x)
    for e in range(layer.experts):
        f = p[f"W2.{e}"].shape[0]
        GU = Y @ p[f"W1.{e}"]
        out = (torch.nn.functional.silu(GU[:, :f]) * GU[:, f:]) @ p[f"W2.{e}"]
        Z = Z + ((ids == e) * weights).sum(-1, keepdim=True) * out
    H = norm(Z + x, p["w2"])
    loss = torch.nn.functional.cross_entropy(H @ p["E"][:layer.vocab].T, targets.long())
    loss.backward()
    return float(loss.detach()), {n: v.grad for n, v in p.items()}


def test_gradients_of_the_expert_layer():
    gpu_or_skip()
    import expert_layer
    layer = expert_layer.ExpertLayer(h=136, f=128, experts=5, k=2, vocab=300, seed=3)
    g = torch.Generator(device="cuda").manual_seed(4)
    S = torch.randn(333, 136, generator=g, device="cuda").to(torch.bfloat16)
    targets = torch.randint(0, 300, (333,), generator=g, device="cuda", dtype=torch.int32)
    loss, grads, ids, _ = layer.loss_and_gradients(S, targets)
    want_loss, want = reference(layer, S, targets, ids)
    assert abs(float(loss) - want_loss) < 1e-2
    assert set(grads) == set(want)
    for n, w in want.items():
        off = float((grads[n].to(D) - w).norm() / w.norm())
        assert off < 2.5e-2, (n, off)


@pytest.mark.parametrize("bits", [8, 32])
def test_training_memorises(bits):
    gpu_or_skip()
    import expert_layer
    losses, kept, packed = expert_layer.train(steps=40, bits=bits)
    assert all(x == x for x in losses)
    assert losses[-1] < losses[0] - 1.0, (losses[0], losses[-1])
    # e4m3 moves the hidden states by 2^-4 of a value at most, 2.6% root mean square
    assert abs(kept - packed) < 0.05 * max(1.0, kept), (kept, packed)


def test_calls_that_nothing_waits_between():
    """Each call reads what the one before wrote: the weights that a step has just updated, the rows that a norm
    has just written. A launch that begins while the kernel before it ends must still see all of it."""
    gpu_or_skip()
    T, h, E, k = 96, 1032, 6, 2
    g = torch.Generator(device="cuda").manual_seed(5)
    X0 = torch.randn(T, h, generator=g, device="cuda").to(torch.bfloat16)
    ids = torch.randint(0, E, (T, k), generator=g, device="cuda", dtype=torch.int32)
    gate = torch.rand(T, k, generator=g, device="cuda")

    def run(wait):
        w = torch.ones(h, device="cuda")
        st = tp.adamw_state(w, 8)
        X = X0.clone()
        kept = []
        for step in range(1, 60):
            f = tp.tp_rmsnorm_forward(X, w, X0)
            wait()
            plan = tp.tp_expert_plan(ids, E)
            wait()
            Xs = tp.tp_expert_dispatch_forward(f["Y"], plan)
            wait()
            X = tp.tp_expert_combine_forward(Xs, plan, gate)
            wait()
            b = tp.tp_rmsnorm_backward(X, f["S"], w, f["rstd"], dS=X0)
            wait()
            tp.adamw_step([w], [b["dw"]], [st], lr=1e-2, step=step)
            wait()
            ids.add_(1).remainder_(E)
            kept.append((X.clone(), w.clone()))
        torch.cuda.synchronize()
        return kept
    start = ids.clone()
    slow = run(torch.cuda.synchronize)
    for _ in range(3):
        ids.copy_(start)
        for i, ((a, b), (c, d)) in enumerate(zip(slow, run(lambda: None))):
            assert torch.equal(a, c) and torch.equal(b, d), i
    assert tp.device_status() == 0
