"""One expert layer trained for a few steps with the library's own calls.

The layer is what a transformer block's second half is in a model with experts:

    Y = norm(S; w1), each token's k of E experts by a linear router on Y,
    Z = sum over its experts of weight * SwiGLU_e(Y),
    H = norm(Z + S; w2), loss = cross-entropy of H over the vocabulary.

RMS norm with the residual's addition, the sort by expert and back, the SwiGLU
block on each expert's rows, the fused vocabulary loss, the backward pass of
each, and one AdamW step over all weights (bf16 with fp32 masters; 8-bit states
for the matrices, 32-bit ones for the norms) run on the GPU; only the rows per
expert are read by the host, which calls the block once per expert. After
training the last hidden states are kept in 8 bits and evaluated from there.

    python examples/expert_layer.py
"""

from __future__ import annotations

import os
import sys
from typing import Dict

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import vocab_ce_gb300 as tp  # noqa: E402

ROUTER_COLUMNS = 64  # the linear layer's narrowest output; the experts take the first columns


class ExpertLayer:
    def __init__(self, h: int, f: int, experts: int, k: int, vocab: int, seed: int = 0, bits: int = 8):
        g = torch.Generator(device="cuda").manual_seed(seed)

        def weight(*shape, std=0.02):
            return std * torch.randn(*shape, generator=g, device="cuda")

        self.experts, self.k, self.vocab = experts, k, vocab
        v_pad = tp.pad_vocab(vocab, 1)
        full = {"router": weight(h, ROUTER_COLUMNS), "E": weight(v_pad, h, std=0.05)}
        for e in range(experts):
            full[f"W1.{e}"], full[f"W2.{e}"] = weight(h, 2 * f, std=0.05), weight(f, h, std=0.05)
        self.masters: Dict[str, torch.Tensor] = full
        self.params = {n: x.to(torch.bfloat16) for n, x in full.items()}
        for n in ("w1", "w2"):
            self.params[n] = torch.ones(h, device="cuda")
        self.states = {n: tp.adamw_state(p, bits if p.dim() == 2 else 32) for n, p in self.params.items()}

    def loss_and_gradients(self, S: torch.Tensor, targets: torch.Tensor):
        """The mean loss, every weight's gradient, the experts chosen and the last hidden states."""
        p, E, k = self.params, self.experts, self.k
        T = S.shape[0]
        # forward
        n1 = tp.tp_rmsnorm_forward(S, p["w1"])
        Y = n1["Y"]
        logits = tp.tp_linear_forward(Y, p["router"], 1)[:, :E].float()
        top, ids = logits.topk(k, -1)
        weights = top.softmax(-1).contiguous()
        plan = tp.tp_expert_plan(ids.int(), E)
        Xs = tp.tp_expert_dispatch_forward(Y, plan)
        edges = plan["offsets"].tolist()
        rows = [slice(a, b) for a, b in zip(edges, edges[1:])]
        Ys = torch.empty_like(Xs)
        saved = [tp.tp_swiglu_forward(Xs[r], p[f"W1.{e}"], p[f"W2.{e}"], 1, out={"Z": Ys[r]})
                 for e, r in enumerate(rows)]
        Z = tp.tp_expert_combine_forward(Ys, plan, weights)
        n2 = tp.tp_rmsnorm_forward(Z, p["w2"], R=S)
        ce = tp.vocab_parallel_ce(n2["Y"], p["E"], targets, self.vocab, 1, grad_scale=1.0 / T)
        # backward
        grads = {"E": ce["dE"]}
        b2 = tp.tp_rmsnorm_backward(ce["dH"], n2["S"], p["w2"], n2["rstd"])
        grads["w2"] = b2["dw"]
        c = tp.tp_expert_combine_backward(b2["dX"], Ys, plan, weights)
        dXs = torch.zeros_like(Xs)
        for e, r in enumerate(rows):
            b = tp.tp_swiglu_backward(c["dYs"][r], Xs[r], p[f"W1.{e}"], p[f"W2.{e}"], saved[e]["GU"], saved[e]["Y"], 1,
                                      bias_grads=False, out={"dX": dXs[r]})
            grads[f"W1.{e}"], grads[f"W2.{e}"] = b["dW1"], b["dW2"]
        dw = c["dweights"]
        dtop = weights * (dw - (weights * dw).sum(-1, keepdim=True))
        dlogits = torch.zeros(T, ROUTER_COLUMNS, device=S.device).scatter_(1, ids, dtop).to(S.dtype)
        r = tp.tp_linear_backward(dlogits, Y, p["router"], 1, bias_grad=False)
        grads["router"] = r["dW"]
        dY = tp.tp_expert_dispatch_backward(dXs, plan) + r["dX"]
        grads["w1"] = tp.tp_rmsnorm_backward(dY, S, p["w1"], n1["rstd"], dS=b2["dX"])["dw"]
        return ce["loss"].mean(), grads, ids, n2

    def update(self, grads: Dict[str, torch.Tensor], step: int, lr: float, weight_decay: float = 0.01) -> None:
        names = list(self.params)
        tp.adamw_step([self.params[n] for n in names], [grads[n] for n in names], [self.states[n] for n in names],
                      lr=lr, step=step, weight_decay=[weight_decay if self.params[n].dim() == 2 else 0.0 for n in names],
                      masters=[self.masters.get(n) for n in names],
                      rounding="random")  # of the 8-bit states: beta2 is 0.999


def train(steps: int = 40, T: int = 1024, h: int = 256, f: int = 512, experts: int = 8, k: int = 2, vocab: int = 1000,
          lr: float = 3e-3, bits: int = 8, seed: int = 0):
    """The losses of the steps, and the last one's from hidden states kept in bf16 and in 8 bits."""
    layer = ExpertLayer(h, f, experts, k, vocab, seed, bits)
    g = torch.Generator(device="cuda").manual_seed(seed + 1)
    S = torch.randn(T, h, generator=g, device="cuda").to(torch.bfloat16)
    targets = torch.randint(0, vocab, (T,), generator=g, device="cuda", dtype=torch.int32)
    losses = []
    for step in range(1, steps + 1):
        loss, grads, _, _ = layer.loss_and_gradients(S, targets)
        layer.update(grads, step, lr)
        losses.append(loss)
    _, _, _, n2 = layer.loss_and_gradients(S, targets)
    # the hidden states in 8 bits, as a cache of features would keep them
    q = tp.tp_rmsnorm_forward(n2["S"], layer.params["w2"], quantize=True, want_Y=False)
    H = (q["Q"].float() * q["Q_scale"].repeat_interleave(128, 1)[:, :h]).to(torch.bfloat16)

    def evaluate(x):
        return float(tp.vocab_parallel_ce(x, layer.params["E"], targets, vocab, 1, grads=False)["loss"].mean())
    return [float(x) for x in losses], evaluate(n2["Y"]), evaluate(H)


if __name__ == "__main__":
    for bits in (32, 8):
        losses, kept, packed = train(bits=bits)
        print(f"AdamW states in {bits} bits: loss {losses[0]:.4f} -> {losses[-1]:.4f}; evaluated from bf16 hidden "
              f"states {kept:.4f}, from 8-bit ones {packed:.4f}")
