"""AdamW with 8-bit states over many steps, beside the same run with 32-bit
states: how large a step may become, and how far a root may lag."""

import math

import pytest
import torch

import vocab_ce_gb300 as tp
from _parity import gpu_or_skip

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
LEAST = 2.0 ** -9   # the smallest code


def generator(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def largest_step(bits, size, decades, steps=400, groups=500):
    """In units of lr: gradients present one step in twenty, their sizes spread inside every group."""
    g, n = generator(0), groups * 128
    sizes = size * 10.0 ** (-decades * torch.rand(n, generator=g, device="cuda"))
    p = torch.zeros(n, device="cuda")
    st, most = tp.adamw_state(p, bits), torch.zeros((), device="cuda")
    for t in range(1, steps + 1):
        there = torch.rand(n, generator=g, device="cuda") < 0.05
        grad = torch.where(there, sizes * torch.randn(n, generator=g, device="cuda"), 0.0)
        p.zero_()
        tp.adamw_step([p], [grad], [st], lr=1.0, step=t)
        most = torch.maximum(most, p.abs().max())
    return float(most)


@pytest.mark.parametrize("decades", [3, 5])
@pytest.mark.parametrize("size", [1e-3, 1.0, 10.0])
def test_rare_gradients_make_no_huge_steps(size, decades):
    """AdamW does not see the gradients' size. A moment that no longer has a gradient stops shrinking at codes of up to
    4.5 smallest ones (0.9 of them rounds to themselves) and its root is at least one: the step is then up to 4.5 times
    the ratio of the group's largest moment and root, which 32-bit states bound."""
    gpu_or_skip()
    assert largest_step(8, size, decades) <= 5.0 * largest_step(32, size, decades)


@pytest.mark.parametrize("p_dtype,master", [(F32, False), (BF, False), (BF, True)])
@pytest.mark.parametrize("n", [1, 128, 300, 2048 + 5])
def test_a_root_that_is_not_zero_keeps_a_code(n, p_dtype, master):
    gpu_or_skip()
    p32 = torch.randn(n, generator=generator(1), device="cuda")
    grad = torch.zeros(n, device="cuda")
    grad[0::128] = 1.0                       # each group's largest
    grad[1::128], grad[2::128], grad[5::128] = 1e-7, -1e-12, float("nan")
    p, st = p32.to(p_dtype), tp.adamw_state(p32, 8)
    tp.adamw_step([p], [grad], [st], lr=1e-3, step=1, masters=[p32.clone()] if master else None)
    r, nan = st["r_q"].float(), grad.isnan()
    assert torch.equal(r.isnan(), nan)
    assert bool((r[0::128] == 448.0).all())
    small = (grad != 0) & ~nan
    small[0::128] = False
    assert bool((r[small] == LEAST).all())   # 1e-7 / 1 and 1e-12 / 1 of 448, below half the smallest code
    assert bool((r[grad == 0] == 0.0).all())
    # a group of zeros, and one whose values are all alike
    st, zero = tp.adamw_state(p32, 8), torch.zeros(n, device="cuda")
    tp.adamw_step([p], [zero], [st], lr=1e-3, step=1)
    assert not st["r_q"].float().any()
    tp.adamw_step([p], [zero + 1e-15], [st], lr=1e-3, step=2)
    assert bool((st["r_q"].float() == 448.0).all()) and math.isclose(float(st["r_scale"][0]) * 448.0,
                                                                     1e-15 * math.sqrt(1 - 0.999), rel_tol=1e-5)
