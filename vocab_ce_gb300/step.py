"""The operators of a training step around the GEMMs: RMS norm with the
residual's addition, tokens sorted by expert and back, and the AdamW step.

Argument marshalling only, as in ``api.py``; the arithmetic is in
``csrc/step/``. With ``stream`` given, new outputs and workspaces are taken
from that stream's memory, and the tensors passed in are recorded on it, so
that memory freed while the stream still works is not handed out again.
Ordering the stream against the ones that made the inputs, or use the outputs,
is the caller's, as with any kernel.
"""

from __future__ import annotations

import ctypes
import math
import struct
from typing import Dict, List, Optional, Sequence, Union

import torch

from ._lib import AdamwTensor, check, lib
from .api import _DT, _need, _workspace, _wsize

GROUP = 128  # values that share one scale in the 8-bit formats
_E4M3 = torch.float8_e4m3fn


# The smallest calls take a few microseconds on the GPU, so the host's part is kept short: the current stream's
# handle without a Stream object around it, plain integers for pointers, and one test for a fitting tensor.
def _current() -> int:
    return torch._C._cuda_getCurrentRawStream(torch.cuda.current_device())


def _handle(stream) -> int:
    return _current() if stream is None else stream.cuda_stream


def _ptr(x: Optional[torch.Tensor]):
    return None if x is None else x.data_ptr()


class _On:
    """Allocations of the launching stream, with the call's tensors recorded on it."""

    __slots__ = ("ctx",)

    def __init__(self, stream, *tensors):
        self.ctx = None
        if stream is not None and stream.cuda_stream != _current():
            for x in tensors:
                if x is not None:
                    x.record_stream(stream)
            self.ctx = torch.cuda.stream(stream)

    def __enter__(self):
        if self.ctx is not None:
            self.ctx.__enter__()

    def __exit__(self, *exc):
        if self.ctx is not None:
            self.ctx.__exit__(*exc)


def _fit(x: torch.Tensor, name: str, dtype, shape, dev: torch.device):
    """x is a contiguous tensor of this type and shape on `dev` (checked to be the current device)."""
    if x.dtype is not dtype or x.shape != shape or x.device != dev or not x.is_contiguous():
        _need(x, name, dtype, shape)


def _dtype(x: torch.Tensor, name: str) -> int:
    dt = _DT.get(x.dtype)
    if dt is None:
        raise ValueError(f"{name} must be torch.bfloat16 or torch.float32, got {x.dtype}")
    return dt


def _matrix(x: torch.Tensor, name: str):
    if x.dim() != 2:
        raise ValueError(f"{name} must be a matrix of rows, got shape {tuple(x.shape)}")
    return x.shape


def _out(out, key, shape, dtype, dev) -> torch.Tensor:
    x = out.get(key) if out else None
    if x is None:
        return torch.empty(shape, dtype=dtype, device=dev)
    _fit(x, key, dtype, shape, dev)
    return x


def _given(out):
    return tuple(out.values()) if out else ()


# ---------------------------------------------------------------------- RMS norm
def rmsnorm_workspace_bytes(T: int, h: int) -> int:
    return int(lib().tpce_rmsnorm_workspace_bytes(T, h))


def tp_rmsnorm_forward(X: torch.Tensor, w: torch.Tensor, R: Optional[torch.Tensor] = None, eps: float = 1e-6,
                       quantize: bool = False, want_Y: bool = True, out: Optional[Dict[str, torch.Tensor]] = None,
                       stream=None) -> Dict[str, torch.Tensor]:
    """S = X + R, rstd = (mean(S^2) + eps)^-1/2, Y = S rstd w; returns Y, rstd,
    with R also S (``out={"S": R}``: in place), and with quantize Q (e4m3) and
    Q_scale, one scale per 128 columns of a row: Y ~ Q * Q_scale."""
    T, h = _matrix(X, "X")
    dt, dev = X.dtype, X.device
    code = _dtype(X, "X")
    _need(X, "X")
    _fit(w, "w", torch.float32, (h,), dev)
    if R is not None:
        _fit(R, "R", dt, X.shape, dev)
    if not (want_Y or quantize):
        raise ValueError("tp_rmsnorm_forward: want_Y or quantize")
    res: Dict[str, torch.Tensor] = {}
    with _On(stream, X, w, R, *_given(out)):
        if R is not None:
            res["S"] = _out(out, "S", (T, h), dt, dev)
        if want_Y:
            res["Y"] = _out(out, "Y", (T, h), dt, dev)
        res["rstd"] = _out(out, "rstd", (T,), torch.float32, dev)
        if quantize:
            res["Q"] = _out(out, "Q", (T, h), _E4M3, dev)
            res["Q_scale"] = _out(out, "Q_scale", (T, -(-h // GROUP)), torch.float32, dev)
    st = lib().tp_rmsnorm_forward(_ptr(X), _ptr(R), _ptr(w), T, h, eps, code, _ptr(res.get("S")), _ptr(res.get("Y")),
                                  _ptr(res.get("Q")), _ptr(res.get("Q_scale")), _ptr(res["rstd"]), _handle(stream))
    check(st, "tp_rmsnorm_forward")
    return res


def tp_rmsnorm_backward(dY: torch.Tensor, S: torch.Tensor, w: torch.Tensor, rstd: torch.Tensor,
                        dS: Optional[torch.Tensor] = None, want_dw: bool = True,
                        out: Optional[Dict[str, torch.Tensor]] = None, ws: Optional[torch.Tensor] = None,
                        stream=None) -> Dict[str, torch.Tensor]:
    """dX, the gradient of X and of R (dS: the gradient that reaches S by the
    residual path), and dw. S is the forward's (X itself where there was no R)."""
    T, h = _matrix(S, "S")
    dt, dev = S.dtype, S.device
    code = _dtype(S, "S")
    _need(S, "S")
    _fit(dY, "dY", dt, S.shape, dev)
    _fit(w, "w", torch.float32, (h,), dev)
    _fit(rstd, "rstd", torch.float32, (T,), dev)
    if dS is not None:
        _fit(dS, "dS", dt, S.shape, dev)
    with _On(stream, dY, S, w, rstd, dS, ws, *_given(out)):
        res = {"dX": _out(out, "dX", (T, h), dt, dev)}
        wk = None
        if want_dw:
            res["dw"] = _out(out, "dw", (h,), torch.float32, dev)
            wk = _workspace(rmsnorm_workspace_bytes(T, h), dev, ws)
    st = lib().tp_rmsnorm_backward(_ptr(dY), _ptr(S), _ptr(w), _ptr(rstd), _ptr(dS), T, h, code, _ptr(res["dX"]),
                                   _ptr(res.get("dw")), _ptr(wk), _wsize(wk), _handle(stream))
    check(st, "tp_rmsnorm_backward")
    return res


# ---------------------------------------------------------------------- experts
def tp_expert_plan(ids: torch.Tensor, experts: int, out: Optional[Dict[str, torch.Tensor]] = None,
                   stream=None) -> Dict[str, torch.Tensor]:
    """The stable sort of the assignments ids [T, k] (int32, -1: dropped) by
    expert: row [T, k], source [T k], offsets [experts + 1], all int32."""
    T, k = _matrix(ids, "ids")
    _need(ids, "ids", torch.int32)
    if experts < 1:
        raise ValueError("experts must be at least 1")
    dev = ids.device
    with _On(stream, ids, *_given(out)):
        res = {"row": _out(out, "row", (T, k), torch.int32, dev),
               "source": _out(out, "source", (T * k,), torch.int32, dev),
               "offsets": _out(out, "offsets", (experts + 1,), torch.int32, dev)}
    check(lib().tp_expert_plan(_ptr(ids), T, k, experts, _ptr(res["row"]), _ptr(res["source"]), _ptr(res["offsets"]),
                               _handle(stream)), "tp_expert_plan")
    return res


def _plan(plan: Dict[str, torch.Tensor]):
    row, offsets = plan["row"], plan["offsets"]
    T, k = _matrix(row, "plan['row']")
    _need(row, "plan['row']", torch.int32)
    if offsets.dim() != 1 or offsets.shape[0] < 2:
        raise ValueError("plan['offsets'] must hold experts + 1 values")
    _fit(offsets, "plan['offsets']", torch.int32, offsets.shape, row.device)
    return row, offsets, T, k, offsets.shape[0] - 1


def tp_expert_dispatch_forward(X: torch.Tensor, plan: Dict[str, torch.Tensor], out: Optional[torch.Tensor] = None,
                               stream=None) -> torch.Tensor:
    """Xs [T k, h]: every kept assignment's copy of its token's row, by expert;
    rows from offsets[experts] on are zeros."""
    row, offsets, T, k, E = _plan(plan)
    code = _dtype(X, "X")
    h = _matrix(X, "X")[1]
    _fit(X, "X", X.dtype, (T, h), row.device)
    with _On(stream, X, row, offsets, out):
        Xs = _out({"Xs": out}, "Xs", (T * k, h), X.dtype, X.device)
    check(lib().tp_expert_dispatch_forward(_ptr(X), _ptr(row), _ptr(offsets), T, h, k, E, code, _ptr(Xs),
                                           _handle(stream)), "tp_expert_dispatch_forward")
    return Xs


def tp_expert_dispatch_backward(dXs: torch.Tensor, plan: Dict[str, torch.Tensor],
                                out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """dX [T, h]: each token's sum over its kept copies."""
    row, _, T, k, _ = _plan(plan)
    code = _dtype(dXs, "dXs")
    h = _matrix(dXs, "dXs")[1]
    _fit(dXs, "dXs", dXs.dtype, (T * k, h), row.device)
    with _On(stream, dXs, row, out):
        dX = _out({"dX": out}, "dX", (T, h), dXs.dtype, dXs.device)
    check(lib().tp_expert_dispatch_backward(_ptr(dXs), _ptr(row), T, h, k, code, _ptr(dX), _handle(stream)),
          "tp_expert_dispatch_backward")
    return dX


def tp_expert_combine_forward(Ys: torch.Tensor, plan: Dict[str, torch.Tensor], weights: torch.Tensor,
                              out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """Z [T, h]: each token's rows of Ys [T k, h], weighted by weights [T, k] (fp32)."""
    row, _, T, k, _ = _plan(plan)
    code = _dtype(Ys, "Ys")
    h = _matrix(Ys, "Ys")[1]
    _fit(Ys, "Ys", Ys.dtype, (T * k, h), row.device)
    _fit(weights, "weights", torch.float32, row.shape, row.device)
    with _On(stream, Ys, row, weights, out):
        Z = _out({"Z": out}, "Z", (T, h), Ys.dtype, Ys.device)
    check(lib().tp_expert_combine_forward(_ptr(Ys), _ptr(row), _ptr(weights), T, h, k, code, _ptr(Z),
                                          _handle(stream)), "tp_expert_combine_forward")
    return Z


def tp_expert_combine_backward(dZ: torch.Tensor, Ys: torch.Tensor, plan: Dict[str, torch.Tensor],
                               weights: torch.Tensor, out: Optional[Dict[str, torch.Tensor]] = None,
                               stream=None) -> Dict[str, torch.Tensor]:
    """dYs [T k, h] (zeros from offsets[experts] on) and dweights [T, k] (fp32, 0 where dropped)."""
    row, offsets, T, k, E = _plan(plan)
    code = _dtype(dZ, "dZ")
    h = _matrix(dZ, "dZ")[1]
    _fit(dZ, "dZ", dZ.dtype, (T, h), row.device)
    _fit(Ys, "Ys", dZ.dtype, (T * k, h), row.device)
    _fit(weights, "weights", torch.float32, row.shape, row.device)
    with _On(stream, dZ, Ys, row, offsets, weights, *_given(out)):
        res = {"dYs": _out(out, "dYs", (T * k, h), dZ.dtype, dZ.device),
               "dweights": _out(out, "dweights", (T, k), torch.float32, dZ.device)}
    check(lib().tp_expert_combine_backward(_ptr(dZ), _ptr(Ys), _ptr(row), _ptr(offsets), _ptr(weights), T, h, k, E,
                                           code, _ptr(res["dYs"]), _ptr(res["dweights"]), _handle(stream)),
          "tp_expert_combine_backward")
    return res


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
        return torch.zeros(param.shape, dtype=torch.uint8, device=param.device).view(_E4M3)

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


_FIELDS = "7QqdiiiI"  # tpce_adamw_tensor
assert struct.calcsize("=" + _FIELDS) == ctypes.sizeof(AdamwTensor)


def _pointers(name: str, xs: Sequence[torch.Tensor], dtype, shapes, dev) -> List[int]:
    """The addresses of contiguous tensors of these shapes on device `dev`; dtype None: bf16 or fp32."""
    for i, x in enumerate(xs):
        if ((x.dtype is not dtype if dtype is not None else x.dtype not in _DT) or x.shape != shapes[i]
                or x.get_device() != dev or not x.is_contiguous()):
            if dtype is None:
                _dtype(x, f"{name}[{i}]")
            _need(x, f"{name}[{i}]", dtype, shapes[i])
    return list(map(torch.Tensor.data_ptr, xs))


def adamw_step(params: Sequence[torch.Tensor], grads: Sequence[torch.Tensor],
               states: Sequence[Dict[str, torch.Tensor]], lr: float, step: int, beta1: float = 0.9,
               beta2: float = 0.999, eps: float = 1e-8, weight_decay: Union[float, Sequence[float]] = 0.0,
               grad_scale: float = 1.0, masters: Optional[Sequence[Optional[torch.Tensor]]] = None,
               scalars: Optional[torch.Tensor] = None, stream=None) -> None:
    """One AdamW step over all tensors, in place: params (fp32 or bf16), their
    fp32 masters where given (then the bf16 parameter is the master's rounding),
    and states (``adamw_state``; the two kinds may mix). step counts from 1.
    scalars: an fp32 tensor of four on the device (``adamw_scalars``) that
    replaces lr, step and grad_scale, for steps captured into a graph."""
    n = len(params)
    if masters is None:
        masters = [None] * n
    decay: List[float] = list(weight_decay) if isinstance(weight_decay, (list, tuple)) else [float(weight_decay)] * n
    for name, x in (("grads", grads), ("states", states), ("masters", masters), ("weight_decay", decay)):
        if len(x) != n:
            raise ValueError(f"{name}: {n} entries expected, got {len(x)}")
    if scalars is not None:
        _need(scalars, "scalars", torch.float32, (4,))
    dev = torch.cuda.current_device() if torch.cuda.is_available() else None
    f32 = torch.float32
    held = [i for i, x in enumerate(masters) if x is not None]
    for i in held:
        if params[i].dtype is f32:
            raise ValueError(f"masters[{i}]: params[{i}] is fp32 already")
    shapes = [p.shape for p in params]
    sizes = [p.numel() for p in params]
    row = [0] * (13 * n)  # the fields of tensor i from 13 i on
    row[0::13] = pp = _pointers("params", params, None, shapes, dev)
    row[2::13] = _pointers("grads", grads, None, shapes, dev)
    row[7::13], row[8::13] = sizes, decay
    row[9::13], row[10::13] = [_DT[p.dtype] for p in params], [_DT[g.dtype] for g in grads]
    if held:
        for i, a in zip(held, _pointers("masters", [masters[i] for i in held], f32, [shapes[i] for i in held], dev)):
            row[13 * i + 1] = a
    # the two kinds of states, each with its places in the list
    for bits in (32, 8):
        at = [i for i, st in enumerate(states) if ("m" in st) == (bits == 32)]
        if not at:
            continue
        full = shapes if len(at) == n else [shapes[i] for i in at]
        few = [(-(-sizes[i] // GROUP),) for i in at]
        parts = (("m", f32, full, 3), ("v", f32, full, 4)) if bits == 32 else (
            ("m_q", _E4M3, full, 3), ("r_q", _E4M3, full, 4), ("m_scale", f32, few, 5), ("r_scale", f32, few, 6))
        for key, dtype, sh, field in parts:
            got = _pointers(key, [states[i][key] for i in at], dtype, sh, dev)
            if len(at) == n:
                row[field::13] = got
            else:
                for i, a in zip(at, got):
                    row[13 * i + field] = a
        if len(at) == n:
            row[11::13] = [bits] * n
        else:
            for i in at:
                row[13 * i + 11] = bits
    if len(set(pp)) != n and len({a for a in pp if a}) != sum(1 for a in pp if a):
        raise ValueError("params: a tensor is in the list twice")
    if stream is not None:
        _On(stream, scalars, *params, *grads, *masters, *(x for st in states for x in st.values()))
    buf = bytearray(ctypes.sizeof(AdamwTensor) * n)
    struct.pack_into("=" + _FIELDS * n, buf, 0, *row)
    tensors = (AdamwTensor * n).from_buffer(buf) if n else None
    check(lib().tp_adamw_step(tensors, n, lr, beta1, beta2, eps, step, grad_scale, _ptr(scalars), _handle(stream)),
          "tp_adamw_step")
