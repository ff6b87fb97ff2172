"""The operators of a training step around the GEMMs: RMS norm with the
residual's addition, tokens sorted by expert and back, the embedding, the
attention core, and the AdamW step.

The arithmetic is in ``csrc/step/*.cu`` and ``csrc/attn/*.cu``; the checks of tensors, the outputs and
the calls of the C ABI are compiled too (``csrc/step/binding.cpp``), because in
Python they would take several times as long as the smallest kernels. With
``stream`` given, new outputs and workspaces are taken from that stream's
memory, and the tensors passed in are recorded on it, so that memory freed
while the stream still works is not handed out again. Ordering the stream
against the ones that made the inputs, or use the outputs, is the caller's, as
with any kernel. The library's pointers are 16-byte aligned; the embedding's ids
and the attention core's offsets, which may be part of a longer vector, are
copied first where they are not.
"""

from __future__ import annotations

import contextlib
import ctypes
import importlib.util
import math
import os
import threading
from typing import Dict, Optional, Sequence, Union

import torch

from ._lib import check, lib
from .build import binding_path

GROUP = 128  # values that share one scale in the 8-bit formats

# the library's entry points that the binding calls, in its order
_ENTRIES = ("tpce_rmsnorm_workspace_bytes", "tp_rmsnorm_forward", "tp_rmsnorm_backward",
            "tpce_expert_plan_workspace_bytes", "tp_expert_plan", "tp_expert_dispatch_forward",
            "tp_expert_dispatch_backward", "tp_expert_combine_forward", "tp_expert_combine_backward", "tp_adamw_step",
            "tpce_embedding_workspace_bytes", "tp_embedding_forward", "tp_embedding_backward",
            "tpce_attn_core_workspace_bytes", "tp_attn_core_forward", "tp_attn_core_backward")
_lock = threading.Lock()
_binding = None


def _b():
    """The loaded binding; raises if it has not been built."""
    return _binding or _load()


def _load():
    global _binding
    with _lock:
        if _binding is None:
            path = binding_path()
            if not os.path.exists(path):
                raise RuntimeError(f"the step binding is not built for this torch and Python ({path}); run "
                                   "`python -m vocab_ce_gb300.build`")
            spec = importlib.util.spec_from_file_location("_step_binding", path)
            module = importlib.util.module_from_spec(spec)
            spec.loader.exec_module(module)
            library = lib()
            module.init(check, torch.OutOfMemoryError,
                        *(ctypes.cast(getattr(library, name), ctypes.c_void_p).value for name in _ENTRIES))
            _binding = module
    return _binding


def _tensors(*xs):
    for x in xs:
        if isinstance(x, torch.Tensor):
            yield x
        elif isinstance(x, dict):
            yield from _tensors(*x.values())
        elif isinstance(x, (list, tuple)):
            yield from _tensors(*x)


def _on(stream, *xs):
    """`stream` as the current one, with the call's tensors recorded on it."""
    if stream.cuda_stream == torch.cuda.current_stream().cuda_stream:
        return contextlib.nullcontext()
    for x in _tensors(*xs):
        if x.is_cuda:
            x.record_stream(stream)
    return torch.cuda.stream(stream)


# ---------------------------------------------------------------------- RMS norm
def rmsnorm_workspace_bytes(T: int, h: int) -> int:
    return int(lib().tpce_rmsnorm_workspace_bytes(T, h))


def tp_rmsnorm_forward(X: torch.Tensor, w: torch.Tensor, R: Optional[torch.Tensor] = None, eps: float = 1e-6,
                       quantize: bool = False, want_Y: bool = True, out: Optional[Dict[str, torch.Tensor]] = None,
                       stream=None) -> Dict[str, torch.Tensor]:
    """S = X + R, rstd = (mean(S^2) + eps)^-1/2, Y = S rstd w; returns Y, rstd,
    with R also S (``out={"S": R}``: in place), and with quantize Q (e4m3) and
    Q_scale, one scale per 128 columns of a row: Y ~ Q * Q_scale."""
    if stream is not None:
        with _on(stream, X, w, R, out):
            return _b().rmsnorm_forward(X, w, R, eps, quantize, want_Y, out)
    return _b().rmsnorm_forward(X, w, R, eps, quantize, want_Y, out)


def tp_rmsnorm_backward(dY: torch.Tensor, S: torch.Tensor, w: torch.Tensor, rstd: torch.Tensor,
                        dS: Optional[torch.Tensor] = None, want_dw: bool = True,
                        out: Optional[Dict[str, torch.Tensor]] = None, ws: Optional[torch.Tensor] = None,
                        stream=None) -> Dict[str, torch.Tensor]:
    """dX, the gradient of X and of R (dS: the gradient that reaches S by the
    residual path), and dw. S is the forward's (X itself where there was no R)."""
    if stream is not None:
        with _on(stream, dY, S, w, rstd, dS, out, ws):
            return _b().rmsnorm_backward(dY, S, w, rstd, dS, want_dw, out, ws)
    return _b().rmsnorm_backward(dY, S, w, rstd, dS, want_dw, out, ws)


# ---------------------------------------------------------------------- experts
def expert_plan_workspace_bytes(T: int, k: int, experts: int) -> int:
    return int(lib().tpce_expert_plan_workspace_bytes(T, k, experts))


def tp_expert_plan(ids: torch.Tensor, experts: int, out: Optional[Dict[str, torch.Tensor]] = None,
                   ws: Optional[torch.Tensor] = None, stream=None) -> Dict[str, torch.Tensor]:
    """The stable sort of the assignments ids [T, k] (int32, -1: dropped) by
    expert: row [T, k], source [T k], offsets [experts + 1], all int32."""
    if stream is not None:
        with _on(stream, ids, out, ws):
            return _b().expert_plan(ids, experts, out, ws)
    return _b().expert_plan(ids, experts, out, ws)


def tp_expert_dispatch_forward(X: torch.Tensor, plan: Dict[str, torch.Tensor], out: Optional[torch.Tensor] = None,
                               stream=None) -> torch.Tensor:
    """Xs [T k, h]: every kept assignment's copy of its token's row, by expert;
    rows from offsets[experts] on are zeros."""
    if stream is not None:
        with _on(stream, X, plan, out):
            return _b().expert_dispatch_forward(X, plan, out)
    return _b().expert_dispatch_forward(X, plan, out)


def tp_expert_dispatch_backward(dXs: torch.Tensor, plan: Dict[str, torch.Tensor],
                                out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """dX [T, h]: each token's sum over its kept copies."""
    if stream is not None:
        with _on(stream, dXs, plan, out):
            return _b().expert_dispatch_backward(dXs, plan, out)
    return _b().expert_dispatch_backward(dXs, plan, out)


def tp_expert_combine_forward(Ys: torch.Tensor, plan: Dict[str, torch.Tensor], weights: torch.Tensor,
                              out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """Z [T, h]: each token's rows of Ys [T k, h], weighted by weights [T, k] (fp32)."""
    if stream is not None:
        with _on(stream, Ys, plan, weights, out):
            return _b().expert_combine_forward(Ys, plan, weights, out)
    return _b().expert_combine_forward(Ys, plan, weights, out)


def tp_expert_combine_backward(dZ: torch.Tensor, Ys: torch.Tensor, plan: Dict[str, torch.Tensor],
                               weights: torch.Tensor, out: Optional[Dict[str, torch.Tensor]] = None,
                               stream=None) -> Dict[str, torch.Tensor]:
    """dYs [T k, h] (zeros from offsets[experts] on) and dweights [T, k] (fp32, 0 where dropped)."""
    if stream is not None:
        with _on(stream, dZ, Ys, plan, weights, out):
            return _b().expert_combine_backward(dZ, Ys, plan, weights, out)
    return _b().expert_combine_backward(dZ, Ys, plan, weights, out)


# ---------------------------------------------------------------------- embedding
def embedding_workspace_bytes(T: int, h: int, v_pad: int) -> int:
    return int(lib().tpce_embedding_workspace_bytes(T, h, v_pad))


def tp_embedding_forward(ids: torch.Tensor, E: torch.Tensor, v_valid: Optional[int] = None, scale: float = 1.0,
                         out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """X [T, h]: scale times the row of E [v_pad, h] that each of ids [T] (int32)
    names. An id is in [0, v_valid) (default: all rows) or -1, padding, whose row
    is zeros; others count as padding and are reported by ``device_status``."""
    if stream is not None:
        with _on(stream, ids, E, out):
            return _b().embedding_forward(ids, E, v_valid, scale, out)
    return _b().embedding_forward(ids, E, v_valid, scale, out)


def tp_embedding_backward(dX: torch.Tensor, ids: torch.Tensor, v_pad: int, v_valid: Optional[int] = None,
                          scale: float = 1.0, out: Optional[torch.Tensor] = None, accumulate: bool = False,
                          ws: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """dE [v_pad, h]: scale times the sum of dX [T, h] over each id's tokens,
    rows without tokens zero. accumulate: added to ``out`` instead, the dE of
    ``vocab_parallel_ce`` where the table is tied, or of the batches before."""
    if stream is not None:
        with _on(stream, dX, ids, out, ws):
            return _b().embedding_backward(dX, ids, v_pad, v_valid, scale, out, accumulate, ws)
    return _b().embedding_backward(dX, ids, v_pad, v_valid, scale, out, accumulate, ws)


# ---------------------------------------------------------------------- attention core
def attn_core_workspace_bytes(T: int, n_heads: int) -> int:
    return int(lib().tpce_attn_core_workspace_bytes(T, n_heads))


def tp_attn_core_forward(QKV: torch.Tensor, n_heads: int, n_kv_heads: int, offsets: Optional[torch.Tensor] = None,
                         window: int = 0, sinks: int = 0, scale: Optional[float] = None,
                         out: Optional[Dict[str, torch.Tensor]] = None, stream=None) -> Dict[str, torch.Tensor]:
    """Causal attention on the fused rows of ``tp_attn_qkv_forward``: O [T, n_heads d]
    and lse [n_heads, T]. offsets [sequences + 1] (int32): sequence b is the rows
    offsets[b] .. offsets[b + 1] (default: one of all rows); rows of none give
    zeros. With a window, a query sees the last ``window`` keys up to its own and
    the first ``sinks`` of its sequence; window 0: all up to its own. scale
    (default 1 / sqrt(d)) multiplies the scores."""
    if stream is not None:
        with _on(stream, QKV, offsets, out):
            return _b().attn_core_forward(QKV, n_heads, n_kv_heads, offsets, window, sinks, scale, out)
    return _b().attn_core_forward(QKV, n_heads, n_kv_heads, offsets, window, sinks, scale, out)


def tp_attn_core_backward(dO: torch.Tensor, QKV: torch.Tensor, O: torch.Tensor, lse: torch.Tensor, n_heads: int,
                          n_kv_heads: int, offsets: Optional[torch.Tensor] = None, window: int = 0, sinks: int = 0,
                          scale: Optional[float] = None, out: Optional[torch.Tensor] = None,
                          ws: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """dQKV, in QKV's columns: what ``tp_attn_qkv_backward`` takes. QKV, O and lse
    are the forward's, the other arguments the same as there."""
    if stream is not None:
        with _on(stream, dO, QKV, O, lse, offsets, out, ws):
            return _b().attn_core_backward(dO, QKV, O, lse, n_heads, n_kv_heads, offsets, window, sinks, scale, out, ws)
    return _b().attn_core_backward(dO, QKV, O, lse, n_heads, n_kv_heads, offsets, window, sinks, scale, out, ws)


# ---------------------------------------------------------------------- AdamW
def adamw_state(param: torch.Tensor, bits: int = 32) -> Dict[str, torch.Tensor]:
    """A tensor's zero state: m and v in fp32, or m_q, m_scale, r_q, r_scale, the
    moment and the root of the second one in e4m3 with a scale per 128 values."""
    if bits == 32:
        return {"m": torch.zeros(param.shape, dtype=torch.float32, device=param.device),
                "v": torch.zeros(param.shape, dtype=torch.float32, device=param.device)}
    if bits != 8:
        raise ValueError("adamw_state: bits must be 8 or 32")
    groups = -(-param.numel() // GROUP)

    def codes():
        return torch.zeros(param.shape, dtype=torch.uint8, device=param.device).view(torch.float8_e4m3fn)

    def scale():
        return torch.zeros(groups, dtype=torch.float32, device=param.device)

    return {"m_q": codes(), "m_scale": scale(), "r_q": codes(), "r_scale": scale()}


def adamw_scalars(lr: float, step: int, beta1: float = 0.9, beta2: float = 0.999,
                  grad_scale: float = 1.0) -> torch.Tensor:
    """The four fp32 values (on the host) that a captured step reads from its
    ``scalars`` tensor: copy them there before each replay."""
    if step < 1:
        raise ValueError("step counts from 1")
    return torch.tensor([lr / (1.0 - beta1 ** step), 1.0 / math.sqrt(1.0 - beta2 ** step), lr, grad_scale],
                        dtype=torch.float32)


def adamw_step(params: Sequence[torch.Tensor], grads: Sequence[torch.Tensor],
               states: Sequence[Dict[str, torch.Tensor]], lr: float, step: int, beta1: float = 0.9,
               beta2: float = 0.999, eps: float = 1e-8, weight_decay: Union[float, Sequence[float]] = 0.0,
               grad_scale: float = 1.0, masters: Optional[Sequence[Optional[torch.Tensor]]] = None,
               scalars: Optional[torch.Tensor] = None, stream=None, rounding: str = "nearest") -> None:
    """One AdamW step over all tensors, in place: params (fp32 or bf16), their
    fp32 masters where given (then the bf16 parameter is the master's rounding),
    and states (``adamw_state``; the two kinds may mix). step counts from 1.
    weight_decay: a number, or one for each tensor. scalars: an fp32 tensor of
    four on the device (``adamw_scalars``) that replaces lr, step and
    grad_scale, for steps captured into a graph. rounding: of 8-bit states,
    "nearest", or "random" where beta2 is near 1 or beta1 above 15/16. To
    nearest, while its group's largest value stays, a root does not grow with
    its gradients until they are sqrt(((17/16)^2 - beta2) / (1 - beta2)) times
    it (11.4 at 0.999, 1.9 at 0.95), and a moment without gradients stops
    shrinking. Random rounding keeps the values' expectations, and gives the
    same bits for the same arguments."""
    if rounding not in ("nearest", "random"):
        raise ValueError('adamw_step: rounding must be "nearest" or "random"')
    random = rounding == "random"
    if stream is not None:
        # read twice below, which an iterator does not allow
        params, grads, states = list(params), list(grads), list(states)
        masters = None if masters is None else list(masters)
        with _on(stream, params, grads, states, masters, scalars):
            return _b().adamw_step(params, grads, states, masters, weight_decay, lr, step, beta1, beta2, eps,
                                   grad_scale, scalars, random)
    return _b().adamw_step(params, grads, states, masters, weight_decay, lr, step, beta1, beta2, eps, grad_scale,
                           scalars, random)
