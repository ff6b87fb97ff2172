"""The embedding and the attention core where they are used: examples/transformer.py's
gradients against autograd in 64 bits on the same weights, its training run, and the
calls without a wait between them.

Gradients: a path rounds at most 11 intermediates of a layer forward (S, Y, QKV, P, O,
A, S, Y, GU, the activation, Z) and 8 backward (dU, dY, dS, dO, dS of the scores, dQKV,
dY, dS) to bf16, two layers and five more at the ends: 43, each off by at most 2^-8 and
2^-8 / sqrt(3) root mean square of its values; independent ones add in squares:
sqrt(43) 2^-8 / sqrt(3) = 1.5% of the gradient's norm where no sum cancels. The
softmaxes' and the norms' gradients cancel: three times that is allowed in the 2-norm.
In fp32 the projections round their operands to tf32, 2^-11, to which the same count
gives 0.2%, three times that is 0.6%.
"""

import os
import sys

import pytest
import torch

import vocab_ce_gb300 as tp
from _attn_ref import visible
from _parity import gpu_or_skip
from _step_ref import D

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))

pytestmark = pytest.mark.gpu


def reference(model, ids, edges, targets, weight, eps=1e-6):
    p = {n: x.to(D).requires_grad_(True) for n, x in model.params.items()}
    n_q, n_kv, d = model.heads, model.kv_heads, model.d

    def norm(s, w):
        return s * (s.pow(2).mean(-1, keepdim=True) + eps).rsqrt() * w

    S = torch.where(ids[:, None] >= 0, p["E"][ids.clamp_min(0).long()] * model.scale, 0.0)
    T = len(ids)
    for i, (window, sinks) in enumerate(model.windows):
        x = (norm(S, p[f"w1.{i}"]) @ p[f"qkv.{i}"]).reshape(T, n_kv, n_q // n_kv + 2, d)
        parts = []
        for a, b in zip(edges, edges[1:]):
            q = x[a:b, :, :-2].reshape(b - a, n_q, d)
            k, v = (x[a:b, :, j].repeat_interleave(n_q // n_kv, 1) for j in (-2, -1))
            s = torch.einsum("qhd,khd->hqk", q, k) / d ** 0.5
            s = s.masked_fill(~visible(b - a, window, sinks, s.device), -torch.inf)
            parts.append(torch.einsum("hqk,khd->qhd", s.softmax(-1), v).reshape(b - a, n_q * d))
        parts.append(torch.zeros(T - edges[-1], n_q * d, dtype=D, device=S.device))
        S = S + torch.cat(parts) @ p[f"out.{i}"]
        GU = norm(S, p[f"w2.{i}"]) @ p[f"W1.{i}"]
        f = GU.shape[1] // 2
        S = S + (torch.nn.functional.silu(GU[:, :f]) * GU[:, f:]) @ p[f"W2.{i}"]
    logits = norm(S, p["wf"]) @ p["E"][:model.vocab].T
    loss = torch.nn.functional.cross_entropy(logits, targets.long(), reduction="none")
    (loss.sum() * weight).backward()
    return loss.detach(), {n: v.grad for n, v in p.items()}


@pytest.mark.parametrize("dtype,allowed", [(torch.bfloat16, 4.5e-2), (torch.float32, 6e-3)])
@pytest.mark.parametrize("heads,kv_heads,d", [(4, 2, 64), (2, 2, 96), (3, 1, 128)])
def test_gradients_of_the_transformer(heads, kv_heads, d, dtype, allowed):
    gpu_or_skip()
    import transformer
    model = transformer.Transformer(2, 136, heads, kv_heads, d, 192, 300, window=50, sinks=3, seed=3, dtype=dtype)
    ids, offsets, targets = transformer.documents((140, 1, 300), 300, 21, 4)
    loss, grads = model.loss_and_gradients(ids, offsets, targets, 0.25)
    want_loss, want = reference(model, ids, offsets.tolist(), targets, 0.25)
    assert set(grads) == set(want)
    for n, w in want.items():
        off = float((grads[n].to(D) - w).norm() / w.norm())
        assert off < allowed, (n, off)
    assert float((loss.to(D) - want_loss).norm() / want_loss.norm()) < allowed
    assert tp.device_status() == 0


def test_training_runs():
    gpu_or_skip()
    import transformer
    losses = transformer.train(steps=3)
    assert len(losses) == 3 and all(x == x and x < 20.0 for x in losses)


def test_calls_that_nothing_waits_between():
    gpu_or_skip()
    import transformer
    ids, offsets, targets = transformer.documents((90, 200), 250, 7, 5)

    def run(wait):
        model = transformer.Transformer(2, 64, 2, 1, 64, 128, 250, window=30, seed=6)
        kept = []
        names = [n for n in dir(tp) if n.startswith("tp_") or n in ("adamw_step", "vocab_parallel_ce")]
        plain = {n: getattr(tp, n) for n in names}

        def waiting(f):
            def call(*a, **k):
                r = f(*a, **k)
                torch.cuda.synchronize()
                return r
            return call
        try:
            if wait:
                for n, f in plain.items():
                    setattr(tp, n, waiting(f))
            for step in range(1, 12):
                loss, grads = model.loss_and_gradients(ids, offsets, targets, 1.0 / 290)
                model.update(grads, step, 1e-2)
                kept.append((loss.clone(), model.params["E"].clone(), model.params["qkv.1"].clone()))
        finally:
            for n, f in plain.items():
                setattr(tp, n, f)
        torch.cuda.synchronize()
        return kept

    slow = run(True)
    for _ in range(3):
        for i, (a, b) in enumerate(zip(slow, run(False))):
            assert all(torch.equal(x, y) for x, y in zip(a, b)), i
    assert tp.device_status() == 0
