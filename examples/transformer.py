"""A small transformer trained on packed documents with the library's own calls.

From token ids to the loss and back: rows of the embedding table, scaled by the
root of the width; in each layer

    Y = norm(S; w1), attention of Y's heads over its document, S += its projection,
    Y = norm(S; w2), SwiGLU block, S += its result,

with a window of ``window`` tokens and the document's first ``sinks`` ones in
every other layer, all tokens in the rest; the last norm, and the fused
vocabulary loss against the same table (tied: the loss writes the table's
gradient and the embedding's backward adds to it). The documents lie one behind
the other in a batch, which ends in padding: ids of -1, rows of no document. One
AdamW step updates all weights (bf16 with fp32 masters). Nothing but the calls
below runs on the GPU.

    python examples/transformer.py
"""

from __future__ import annotations

import math
import os
import sys
from typing import Dict, Sequence

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import vocab_ce_gb300 as tp  # noqa: E402


class Transformer:
    def __init__(self, layers: int, h: int, heads: int, kv_heads: int, d: int, f: int, vocab: int, window: int = 64,
                 sinks: int = 2, seed: int = 0, dtype: torch.dtype = torch.bfloat16):
        g = torch.Generator(device="cuda").manual_seed(seed)

        def weight(*shape, std):
            return std * torch.randn(*shape, generator=g, device="cuda")

        self.layers, self.heads, self.kv_heads, self.d, self.vocab = layers, heads, kv_heads, d, vocab
        self.windows = [(window, sinks) if i % 2 else (0, 0) for i in range(layers)]
        self.scale = math.sqrt(h)
        self.v_pad = tp.pad_vocab(vocab, 1)
        full = {"E": weight(self.v_pad, h, std=h ** -0.5)}
        norms = ["wf"]
        for i in range(layers):
            full[f"qkv.{i}"] = weight(h, (heads + 2 * kv_heads) * d, std=h ** -0.5)
            full[f"out.{i}"] = weight(heads * d, h, std=(heads * d) ** -0.5 / math.sqrt(2 * layers))
            full[f"W1.{i}"] = weight(h, 2 * f, std=h ** -0.5)
            full[f"W2.{i}"] = weight(f, h, std=f ** -0.5 / math.sqrt(2 * layers))
            norms += [f"w1.{i}", f"w2.{i}"]
        self.masters: Dict[str, torch.Tensor] = full if dtype == torch.bfloat16 else {}
        self.params = {n: x.to(dtype) for n, x in full.items()}
        for n in norms:
            self.params[n] = torch.ones(h, device="cuda")
        self.states = {n: tp.adamw_state(p) for n, p in self.params.items()}

    def loss_and_gradients(self, ids: torch.Tensor, offsets: torch.Tensor, targets: torch.Tensor, weight: float):
        """The tokens' losses and the gradients of `weight` times their sum. ids [T] int32 (-1: padding), offsets of
        the documents, targets [T] int32 in [0, vocab)."""
        p = self.params
        heads = dict(n_heads=self.heads, n_kv_heads=self.kv_heads)
        # forward
        Z = tp.tp_embedding_forward(ids, p["E"], v_valid=self.vocab, scale=self.scale)
        S, saved = None, []
        for i, (window, sinks) in enumerate(self.windows):
            n1 = tp.tp_rmsnorm_forward(Z, p[f"w1.{i}"], R=S)
            S1 = n1.get("S", Z)
            QKV = tp.tp_attn_qkv_forward(n1["Y"], p[f"qkv.{i}"], self.heads, self.kv_heads, self.d, 1)
            core = tp.tp_attn_core_forward(QKV, offsets=offsets, window=window, sinks=sinks, **heads)
            A = tp.tp_attn_out_forward(core["O"], p[f"out.{i}"], self.heads, self.d, 1)
            n2 = tp.tp_rmsnorm_forward(A, p[f"w2.{i}"], R=S1)
            block = tp.tp_swiglu_forward(n2["Y"], p[f"W1.{i}"], p[f"W2.{i}"], 1)
            saved.append((n1, S1, QKV, core, n2, block))
            Z, S = block["Z"], n2["S"]
        last = tp.tp_rmsnorm_forward(Z, p["wf"], R=S)
        ce = tp.vocab_parallel_ce(last["Y"], p["E"], targets, self.vocab, 1, grad_scale=weight)
        # backward
        grads = {}
        b = tp.tp_rmsnorm_backward(ce["dH"], last["S"], p["wf"], last["rstd"])
        grads["wf"], dS = b["dw"], b["dX"]
        for i in reversed(range(self.layers)):
            n1, S1, QKV, core, n2, block = saved[i]
            window, sinks = self.windows[i]
            b = tp.tp_swiglu_backward(dS, n2["Y"], p[f"W1.{i}"], p[f"W2.{i}"], block["GU"], block["Y"], 1,
                                      bias_grads=False)
            grads[f"W1.{i}"], grads[f"W2.{i}"] = b["dW1"], b["dW2"]
            b = tp.tp_rmsnorm_backward(b["dX"], n2["S"], p[f"w2.{i}"], n2["rstd"], dS=dS)
            grads[f"w2.{i}"], dS = b["dw"], b["dX"]
            b = tp.tp_attn_out_backward(dS, core["O"], p[f"out.{i}"], self.heads, self.d, 1, bias_grad=False)
            grads[f"out.{i}"] = b["dWo"]
            dQKV = tp.tp_attn_core_backward(b["dO"], QKV, core["O"], core["lse"], offsets=offsets, window=window,
                                            sinks=sinks, **heads)
            b = tp.tp_attn_qkv_backward(dQKV, n1["Y"], p[f"qkv.{i}"], self.heads, self.kv_heads, self.d, 1,
                                        bias_grad=False)
            grads[f"qkv.{i}"] = b["dWqkv"]
            b = tp.tp_rmsnorm_backward(b["dX"], S1, p[f"w1.{i}"], n1["rstd"], dS=dS)
            grads[f"w1.{i}"], dS = b["dw"], b["dX"]
        grads["E"] = tp.tp_embedding_backward(dS, ids, self.v_pad, v_valid=self.vocab, scale=self.scale, out=ce["dE"],
                                              accumulate=True)
        return ce["loss"], grads

    def update(self, grads: Dict[str, torch.Tensor], step: int, lr: float, weight_decay: float = 0.01) -> None:
        names = list(self.params)
        tp.adamw_step([self.params[n] for n in names], [grads[n] for n in names], [self.states[n] for n in names],
                      lr=lr, step=step, beta2=0.95,
                      weight_decay=[weight_decay if self.params[n].dim() == 2 else 0.0 for n in names],
                      masters=[self.masters.get(n) for n in names])


def documents(lengths: Sequence[int], vocab: int, padding: int, seed: int = 0):
    """Packed documents, each a repeated phrase: ids, offsets, and every token's next one as its target (a
    document's last token, and padding, have the token 0)."""
    g = torch.Generator().manual_seed(seed)
    ids, targets, edges = [], [], [0]
    for n in lengths:
        phrase = torch.randint(1, vocab, (max(2, n // 7),), generator=g)
        text = phrase.repeat(-(-n // len(phrase)))[:n]
        ids.append(text)
        targets.append(torch.cat([text[1:], torch.zeros(1, dtype=text.dtype)]))
        edges.append(edges[-1] + n)
    ids.append(torch.full((padding,), -1))
    targets.append(torch.zeros(padding, dtype=torch.long))
    return (torch.cat(ids).int().cuda(), torch.tensor(edges, dtype=torch.int32, device="cuda"),
            torch.cat(targets).int().cuda())


def train(steps: int = 60, layers: int = 2, h: int = 256, heads: int = 4, kv_heads: int = 2, d: int = 64, f: int = 512,
          vocab: int = 500, lengths: Sequence[int] = (300, 41, 520, 130), padding: int = 33, lr: float = 3e-3,
          seed: int = 0):
    """The mean losses of the documents' tokens, step by step."""
    model = Transformer(layers, h, heads, kv_heads, d, f, vocab, seed=seed)
    ids, offsets, targets = documents(lengths, vocab, padding, seed + 1)
    tokens = sum(lengths)
    losses = []
    for step in range(1, steps + 1):
        loss, grads = model.loss_and_gradients(ids, offsets, targets, 1.0 / tokens)
        model.update(grads, step, lr)
        losses.append(loss[:tokens].mean())
    return [float(x) for x in losses]


if __name__ == "__main__":
    losses = train()
    print("loss " + " -> ".join(f"{losses[i]:.4f}" for i in range(0, len(losses), 10)) + f" -> {losses[-1]:.4f}")
