"""The AdamW step's lists: what they may not hold, and nothing changed where they
are refused."""

import pytest
import torch

import vocab_ce_gb300 as tp
from _parity import gpu_or_skip

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
STEP = dict(lr=1e-3, step=1)


def normal(n, seed, dtype=F32):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(n, generator=g, device="cuda").to(dtype)


@pytest.mark.parametrize("bits", [8, 32])
def test_what_would_be_written_twice_is_refused(bits):
    gpu_or_skip()
    p, q, g, h = normal(300, 1), normal(300, 2), normal(300, 3), normal(300, 4)
    b, c = p.to(BF), q.to(BF)
    st, su = tp.adamw_state(p, bits), tp.adamw_state(q, bits)
    flat, one = normal(1000, 5), tp.adamw_state(normal(600, 6), bits)
    bad = [([p, q], [g, h], [st, st], None),                                        # one state for two
           ([p, q], [g, h], [st, dict(su, **{k: st[k] for k in list(st)[:1]})], None),  # a part of it
           ([b, c], [g, h], [st, su], [p, p]),                                      # one master for two
           ([b, p], [g, h], [st, su], [p, None]),                                   # a master that is a parameter too
           ([flat[:600], flat[320:920]], [normal(600, 7), normal(600, 8)], [one, tp.adamw_state(flat[:600], bits)], None),
           ([p, q], [g, p], [st, su], None)]                                        # a gradient that is a parameter
    if bits == 32:
        bad.append(([p, q], [g, st["m"]], [st, su], None))                          # a gradient that is a moment
    before = [x.clone() for x in (p, q, b, c, flat, *st.values(), *su.values(), *one.values())]
    for params, grads, states, masters in bad:
        with pytest.raises(tp.TpceError, match="overlaps"):
            tp.adamw_step(params, grads, states, masters=masters, **STEP)
    for x, y in zip((p, q, b, c, flat, *st.values(), *su.values(), *one.values()), before):
        assert torch.equal(x.view(torch.uint8), y.view(torch.uint8))
    # one gradient for two parameters, and neighbours in one buffer, are none of these
    tp.adamw_step([p, q], [g, g], [st, su], **STEP)
    tp.adamw_step([flat[:320], flat[320:920]], [normal(320, 9), normal(600, 10)],
                  [tp.adamw_state(flat[:320], bits), one], **STEP)
    assert not torch.equal(p, before[0]) and not torch.equal(flat[:320], before[4][:320])
