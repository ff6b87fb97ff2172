"""The AdamW step's lists: what they may not hold, with nothing changed where they
are refused; lists around the sizes where launches and blocks change, against
elementary 32-bit operations (the same bits)."""

import pytest
import torch

import vocab_ce_gb300 as tp
from _parity import gpu_or_skip
from test_gpu_step_adamw import HYPER, KINDS, copy, elementary, same, step, tensors

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
           ([flat[:600], flat[320:920]], [normal(600, 7), normal(600, 8)],          # neighbours that overlap
            [one, tp.adamw_state(flat[:600], bits)], None),
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


@pytest.mark.parametrize("count", [1, 2, 43, 44, 45, 135, 136, 137, 367, 368, 369, 735, 736, 737])
def test_lists_at_the_ends_of_a_launch_s_tables(count):
    # tables of 44, 136 and 368 tensors; the longest full, one more than it, and a list that ends with a full one
    gpu_or_skip()
    kinds = [(k, b) for k in KINDS for b in (8, 32)]
    old = [tensors(1 + (53 * i) % 400, *kinds[i % 12][0], kinds[i % 12][1], i) for i in range(count)]
    for empty in (False, True):
        many, plain = [copy(t) for t in old], [copy(t) for t in old]
        if empty:   # tensors without values take no place in a table
            many[count // 2:count // 2] = [tensors(0, F32, F32, False, b, 0) for b in (8, 32)]
        step(many)
        for t in plain:
            elementary(t, 0.1)
        for i, (t, q) in enumerate(zip((t for t in many if t["p"].numel()), plain)):
            same(t, q, f"{i} of {count}")


def test_a_list_long_enough_for_blocks_of_several_chunks():
    # from 4864 chunks of 2048 values on, blocks of tensors with 8-bit states take four; ends inside a block's first,
    # second and fourth chunk, at a chunk's and at a block's end, and tensors with 32-bit states between them
    gpu_or_skip()
    chunk = 2048
    sizes = [(2_000_000 + 5, 8), (1_500_003, 32), (4 * chunk * 200, 8), (4 * chunk * 150 + chunk, 8), (700_001, 32),
             (4 * chunk * 170 + 3 * chunk + 1, 8), (4 * chunk * 100 + chunk + 127, 8), (1, 8), (7, 32),
             (3_000_000, 8), (129, 8), (900_000, 32)]
    old = [tensors(n, *KINDS[i % 6], bits, 10 * i) for i, (n, bits) in enumerate(sizes)]
    assert sum(-(-n // chunk) for n, _ in sizes) >= 4864
    many, plain = [copy(t) for t in old], [copy(t) for t in old]
    step(many)
    for t, q, (n, bits) in zip(many, plain, sizes):
        elementary(q, 0.1)
        same(t, q, f"{n} values, {bits} bits")
    for i in (0, 3, 5):     # and as alone, a chunk a block
        t = copy(old[i])
        step([t])
        same(t, many[i])


@pytest.mark.parametrize("own_stream", [False, True])
def test_lists_that_can_be_read_once(own_stream):
    # model.parameters() and the like; with a stream the tensors are recorded on it first
    gpu_or_skip()
    old = [tensors(n, BF, F32, True, 8, n) for n in (300, 77, 4000)]
    one, two = [copy(t) for t in old], [copy(t) for t in old]
    stream = torch.cuda.Stream() if own_stream else None
    if stream is not None:
        stream.wait_stream(torch.cuda.current_stream())
    tp.adamw_step((t["p"] for t in one), (t["g"] for t in one), (t["st"] for t in one),
                  masters=(t["master"] for t in one), weight_decay=(0.1 for t in one), stream=stream, **HYPER)
    if stream is not None:
        torch.cuda.current_stream().wait_stream(stream)
    step(two)
    for t, q, o in zip(one, two, old):
        same(t, q)
        assert not torch.equal(t["master"], o["master"])
