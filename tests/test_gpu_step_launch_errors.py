"""A launch that the runtime turns down: that call fails, and the next does not.

A launch into the legacy stream while a stream that it would wait for captures is
refused on the host (and ends the capture); nothing reaches the GPU."""

import ctypes

import pytest
import torch

import vocab_ce_gb300 as tp
from _parity import gpu_or_skip
from vocab_ce_gb300._lib import lib

pytestmark = pytest.mark.gpu
GLOBAL = 0   # cudaStreamCaptureModeGlobal


def runtime():
    for name in ("libcudart.so.13", "libcudart.so"):
        try:
            return ctypes.CDLL(name)
        except OSError:
            pass
    pytest.skip("no shared CUDA runtime to begin a capture with")


def calls():
    X, w = torch.randn(64, 512, device="cuda"), torch.ones(512, device="cuda")
    n = tp.tp_rmsnorm_forward(X, w)
    dX = torch.empty_like(X)
    ids = torch.randint(0, 4, (64, 2), device="cuda", dtype=torch.int32)
    plan = tp.tp_expert_plan(ids, 4)
    Xs = tp.tp_expert_dispatch_forward(X, plan)
    p, st = X[0].clone(), tp.adamw_state(X[0])
    return {"forward": lambda: tp.tp_rmsnorm_forward(X, w, out=n),
            "backward": lambda: tp.tp_rmsnorm_backward(X, X, w, n["rstd"], want_dw=False, out={"dX": dX}),
            "plan": lambda: tp.tp_expert_plan(ids, 4, out=plan),
            "dispatch": lambda: tp.tp_expert_dispatch_forward(X, plan, out=Xs),
            "adamw": lambda: tp.adamw_step([p], [w], [st], lr=1e-3, step=1),
            "no tokens": lambda: tp.tp_expert_plan(ids[:0], 4)}


@pytest.mark.parametrize("name", ["forward", "backward", "plan", "dispatch", "adamw", "no tokens"])
def test_a_refused_launch_does_not_fail_the_next_call(name):
    gpu_or_skip()
    rt, call = runtime(), calls()[name]
    assert torch.cuda.current_stream().cuda_stream == 0      # the legacy stream
    call()
    torch.cuda.synchronize()
    side, graph = ctypes.c_void_p(), ctypes.c_void_p()
    assert rt.cudaStreamCreate(ctypes.byref(side)) == 0      # a blocking one: torch's own are not
    assert rt.cudaStreamBeginCapture(side, GLOBAL) == 0
    try:
        with pytest.raises(tp.TpceError):
            call()
    finally:
        rt.cudaStreamEndCapture(side, ctypes.byref(graph))
        rt.cudaStreamDestroy(side)
        rt.cudaGetLastError()
    call()
    torch.cuda.synchronize()
    assert tp.device_status() == 0


@pytest.mark.parametrize("name", ["forward", "plan", "adamw"])
def test_what_failed_before_is_not_this_call_s_failure(name):
    gpu_or_skip()
    rt, call = runtime(), calls()[name]
    call()
    torch.cuda.synchronize()
    side, graph = ctypes.c_void_p(), ctypes.c_void_p()
    assert rt.cudaStreamCreate(ctypes.byref(side)) == 0
    assert rt.cudaStreamBeginCapture(side, GLOBAL) == 0
    try:
        # the status word is read after a synchronisation, which a captured stream refuses
        assert lib().tpce_device_status(side, 0, None) == 5
    finally:
        rt.cudaStreamEndCapture(side, ctypes.byref(graph))
        rt.cudaStreamDestroy(side)
        rt.cudaGetLastError()
    call()
    torch.cuda.synchronize()
    assert tp.device_status() == 0
