"""The RMS norm's bounded waits when what they wait for never comes.

tpce_debug_withhold_next_load(1) makes block 0 of the next norm launch whose
rows come through a ring count bytes on its first row that nothing copies: the
wait for that row cannot complete. No fault is involved. For each kernel with a ring the test checks that

* the call returns, after the wait's bound (2 s) and a drain's (50 ms: the block
  may not leave while something is under way to its shared memory), and well
  before any outer limit;
* the device status word names a wait of the norm;
* the context is usable: the same call again gives the bits from before.
"""

import time

import pytest
import torch

import vocab_ce_gb300 as tp
from _parity import gpu_or_skip
from vocab_ce_gb300._lib import lib

pytestmark = pytest.mark.gpu
TIMEOUT = 6
WAIT_ROW, WAIT_SUMS, WAIT_STAGE = 20, 21, 22
WAIT_S, DRAIN_S = 2.0, 0.05


def normal(shape, dtype, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(shape, generator=g, device="cuda").to(dtype)


def forward(T, h, dtype, residual):
    x, w = normal((T, h), dtype, 1), normal((h,), torch.float32, 2)
    r = normal((T, h), dtype, 3) if residual else None
    return lambda: tp.tp_rmsnorm_forward(x, w, R=r, quantize=True)


def backward(T, h, dtype, residual):
    y, s, w = normal((T, h), dtype, 1), normal((T, h), dtype, 2), normal((h,), torch.float32, 3)
    d = normal((T, h), dtype, 4) if residual else None
    rstd = s.float().pow(2).mean(-1).add(1e-6).rsqrt()
    return lambda: tp.tp_rmsnorm_backward(y, s, w, rstd, dS=d)


# every kernel with a ring, one to three tensors a row; more rows than fill the ring once, so that block 0 has fills
# to skip after its wait ran out
CASES = {
    "forward": (forward, 30_000, 1024, torch.bfloat16, False),
    "forward residual": (forward, 3000, 8192, torch.bfloat16, True),
    "forward fp32": (forward, 3000, 4096, torch.float32, False),
    "backward": (backward, 12_000, 1024, torch.bfloat16, True),
    "backward fp32": (backward, 1500, 8192, torch.float32, False),
    "backward pair": (backward, 1500, 16_384, torch.bfloat16, True),
    "backward pair fp32": (backward, 1500, 16_384, torch.float32, True),
}


@pytest.mark.parametrize("name", CASES)
def test_withheld_row_times_out_and_the_context_stays_usable(name):
    gpu_or_skip()
    make, T, h, dtype, residual = CASES[name]
    call = make(T, h, dtype, residual)
    assert tp.device_status(clear=True) == 0
    want = call()
    torch.cuda.synchronize()

    assert lib().tpce_debug_withhold_next_load(1) == 0
    t0 = time.perf_counter()
    call()
    code, detail = tp.device_status_detail(clear=True)   # synchronises the stream
    elapsed = time.perf_counter() - t0
    assert code == TIMEOUT, (code, hex(detail))
    assert (detail >> 8) & 0xff in (WAIT_ROW, WAIT_SUMS, WAIT_STAGE), hex(detail)
    assert WAIT_S + DRAIN_S <= elapsed < 30.0, elapsed

    for _ in range(2):
        got = call()
        assert tp.device_status(clear=True) == 0
        for key, x in want.items():
            assert torch.equal(x.view(torch.uint8), got[key].view(torch.uint8)), key


def test_a_launch_without_a_ring_leaves_the_knob_armed():
    gpu_or_skip()
    small = forward(4, 1024, torch.bfloat16, True)        # a row a block: nothing is fetched ahead
    narrow = backward(4000, 256, torch.bfloat16, False)   # rows of a warp
    assert lib().tpce_debug_withhold_next_load(1) == 0
    small()
    narrow()
    assert tp.device_status(clear=True) == 0
    assert lib().tpce_debug_withhold_next_load(0) == 0
