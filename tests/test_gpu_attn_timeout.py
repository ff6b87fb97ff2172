"""The attention core's bounded waits when what they wait for never comes.

tpce_debug_withhold_next_load(1) makes block 0 of the next bf16 attention launch
load nothing of its first tile of keys (of its first step's tiles in the
backward): the waits for it cannot complete. No fault is involved. The call
returns after the waits' bound (2 s) and a drain's, the status word names a
timeout, and the same call again gives the bits from before. With a number of nanoseconds
the next forward's blocks give up after that time instead, in the middle of their work.
"""

import time

import pytest
import torch

import vocab_ce_gb300 as tp
from _parity import gpu_or_skip
from vocab_ce_gb300._lib import lib

pytestmark = pytest.mark.gpu
TIMEOUT = 6
WAIT_S = 2.0


@pytest.mark.parametrize("T,G,window", [(3000, 2, 0), (700, 1, 200), (50, 4, 0)])
@pytest.mark.parametrize("direction", ["forward", "backward"])
def test_a_tile_that_never_comes(direction, T, G, window):
    gpu_or_skip()
    g = torch.Generator(device="cuda").manual_seed(T)
    QKV = torch.randn(T, (G + 2) * 2 * 64, generator=g, device="cuda").bfloat16()
    dO = torch.randn(T, G * 2 * 64, generator=g, device="cuda").bfloat16()
    f = tp.tp_attn_core_forward(QKV, 2 * G, 2, window=window)

    def call():
        if direction == "forward":
            return tp.tp_attn_core_forward(QKV, 2 * G, 2, window=window)["O"]
        return tp.tp_attn_core_backward(dO, QKV, f["O"], f["lse"], 2 * G, 2, window=window)

    good = call()
    torch.cuda.synchronize()
    assert tp.device_status() == 0
    assert lib().tpce_debug_withhold_next_load(1) == 0
    t0 = time.monotonic()
    call()
    torch.cuda.synchronize()
    took = time.monotonic() - t0
    assert WAIT_S - 0.1 <= took < WAIT_S + 1.0, took
    assert tp.device_status() == TIMEOUT and tp.device_status() == 0
    again = call()
    assert torch.equal(good, again) and tp.device_status() == 0


@pytest.mark.parametrize("T,n_kv,G,window", [(3000, 4, 8, 0), (3000, 16, 1, 500), (90, 1, 2, 0)])
def test_blocks_that_give_up_while_others_get_on(T, n_kv, G, window):
    # two warps share queries: neither may wait for the other when that has left
    gpu_or_skip()
    g = torch.Generator(device="cuda").manual_seed(T)
    QKV = torch.randn(T, (G + 2) * n_kv * 128, generator=g, device="cuda").bfloat16()

    def call():
        f = tp.tp_attn_core_forward(QKV, n_kv * G, n_kv, window=window)
        return f["O"], f["lse"]

    good = call()
    torch.cuda.synchronize()
    assert tp.device_status() == 0
    for k in range(100):
        assert lib().tpce_debug_withhold_next_load(2 + 311 * k) == 0       # up to 31 us
        t0 = time.monotonic()
        call()
        torch.cuda.synchronize()
        took = time.monotonic() - t0
        assert tp.device_status_detail() == (TIMEOUT, TIMEOUT | 29 << 8), k
        assert took < 1.0, (k, took)   # what is given up is not waited for
    again = call()
    assert all(torch.equal(x, y) for x, y in zip(good, again)) and tp.device_status() == 0


def test_a_copy_that_is_given_up_is_waited_for_once_more():
    # its tile ends a sequence, and lands on a barrier of its own: with nothing loaded the wait for what may still be
    # under way takes its whole limit, 50 ms, after the 2 s
    gpu_or_skip()
    g = torch.Generator(device="cuda").manual_seed(1)
    QKV = torch.randn(50, 6 * 64, generator=g, device="cuda").bfloat16()
    dO = torch.randn(50, 4 * 64, generator=g, device="cuda").bfloat16()
    f = tp.tp_attn_core_forward(QKV, 4, 1)
    good = tp.tp_attn_core_backward(dO, QKV, f["O"], f["lse"], 4, 1)
    torch.cuda.synchronize()
    assert lib().tpce_debug_withhold_next_load(1) == 0
    t0 = time.monotonic()
    tp.tp_attn_core_backward(dO, QKV, f["O"], f["lse"], 4, 1)
    torch.cuda.synchronize()
    took = time.monotonic() - t0
    assert WAIT_S + 0.045 <= took < WAIT_S + 1.0, took
    assert tp.device_status() == TIMEOUT
    assert torch.equal(good, tp.tp_attn_core_backward(dO, QKV, f["O"], f["lse"], 4, 1)) and tp.device_status() == 0
