"""Arguments of the training-step calls that Python itself cannot make sense of:
the error is Python's, and nothing has been launched."""

import pytest
import torch

import vocab_ce_gb300 as tp
from _parity import gpu_or_skip

pytestmark = pytest.mark.gpu


class NoTruth:
    def __bool__(self):
        raise KeyError("neither")


def test_a_switch_without_a_truth_value_raises_before_the_launch():
    gpu_or_skip()
    X = torch.ones(4, 64, device="cuda")
    w, rstd = torch.ones(64, device="cuda"), torch.ones(4, device="cuda")
    Y, Q = torch.full_like(X, 7.0), torch.zeros(4, 64, device="cuda").to(torch.float8_e4m3fn)
    for bad in (NoTruth(), torch.zeros(2)):
        for name in ("quantize", "want_Y"):
            with pytest.raises((KeyError, RuntimeError)):
                tp.tp_rmsnorm_forward(X, w, out={"Y": Y, "Q": Q}, **{name: bad})
        with pytest.raises((KeyError, RuntimeError)):
            tp.tp_rmsnorm_backward(X, X, w, rstd, want_dw=bad, out={"dX": Y})
    torch.cuda.synchronize()
    assert bool((Y == 7.0).all()) and not Q.float().any()
