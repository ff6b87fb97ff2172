"""The attention core's refusals and workspace sizes, on the CPU: every call here
is turned down by the library's host checks (the pointers are never read)."""

import ctypes

import pytest

P = ctypes.c_void_p
INVALID, SHAPE, ALIGN, WORKSPACE = 1, 2, 3, 4
MB = 1 << 20


@pytest.fixture(scope="module")
def L():
    from vocab_ce_gb300 import build
    build.build()
    from vocab_ce_gb300._lib import lib
    return lib()


def forward(L, T=100, n=4, kv=2, d=64, window=0, sinks=0, scale=0.125, dtype=0, QKV=MB, offsets=2 * MB, b=3, O=3 * MB,
            lse=4 * MB):
    return L.tp_attn_core_forward(P(QKV), P(offsets), b, T, n, kv, d, window, sinks, scale, dtype, P(O), P(lse), None)


def backward(L, T=100, n=4, kv=2, d=64, window=0, sinks=0, scale=0.125, dtype=0, dO=MB, QKV=2 * MB, O=3 * MB,
             lse=4 * MB, offsets=5 * MB, b=3, dQKV=6 * MB, ws=7 * MB, size=1 << 30):
    return L.tp_attn_core_backward(P(dO), P(QKV), P(O), P(lse), P(offsets), b, T, n, kv, d, window, sinks, scale, dtype,
                                   P(dQKV), P(ws), size, None)


@pytest.mark.parametrize("call", [forward, backward])
def test_shapes(L, call):
    assert call(L, T=0) == 0
    for bad in ({"T": -1}, {"n": 0}, {"kv": 0}, {"n": 3}, {"n": -2, "kv": -1}, {"n": 4098}, {"d": 0}, {"d": 12},
                {"d": 136}, {"window": -1}, {"sinks": -1}, {"b": 0}, {"b": -1}, {"T": (1 << 30) + 1},
                {"T": 1 << 30, "n": 16}, {"T": 1 << 29, "n": 256, "kv": 1}, {"b": 1 << 30}):
        assert call(L, **bad) == SHAPE, bad
    assert call(L, b=-1, offsets=0) == SHAPE
    for bad in ({"dtype": 2}, {"dtype": -1}, {"scale": float("inf")}, {"scale": float("nan")}):
        assert call(L, **bad) == INVALID, bad


@pytest.mark.parametrize("call,names", [(forward, ("QKV", "O", "lse")), (backward, ("dO", "QKV", "O", "lse", "dQKV"))])
def test_pointers(L, call, names):
    for name in names:
        assert call(L, **{name: 0}) == INVALID and call(L, **{name: MB * 8 + 8}) == ALIGN, name
    assert call(L, offsets=2 * MB + 4) == ALIGN


def test_overlaps(L):
    row = 8 * 64 * 2                      # of QKV, in bytes
    for bad in ({"O": MB}, {"O": MB + 99 * row}, {"lse": MB + 16}, {"lse": 3 * MB + 16}, {"lse": 2 * MB},
                {"O": 2 * MB - 16}):
        assert forward(L, **bad) == INVALID and b"overlap" in L.tpce_last_error(), bad
    for bad in ({"dQKV": 2 * MB}, {"dQKV": MB}, {"dQKV": 3 * MB + 16}, {"dQKV": 5 * MB - 16}, {"ws": 6 * MB},
                {"ws": 4 * MB}, {"dQKV": 4 * MB - row}):
        assert backward(L, **bad) == INVALID and b"overlap" in L.tpce_last_error(), bad


def test_workspace(L):
    import vocab_ce_gb300 as tp
    need = tp.attn_core_workspace_bytes
    assert need(0, 4) == 0 and need(-1, 4) == 0 and need(100, 0) == 0
    size = need(100, 4)
    assert size >= 100 * 4 * 8
    assert backward(L, ws=0) == WORKSPACE and backward(L, size=size - 1) == WORKSPACE
    assert str(size) in L.tpce_last_error().decode()
    assert backward(L, ws=7 * MB + 8) == ALIGN


def test_cpu_tensors_are_refused(L):
    torch = pytest.importorskip("torch")
    import vocab_ce_gb300 as tp
    x = torch.zeros(4, 4 * 64)
    with pytest.raises(ValueError):
        tp.tp_attn_core_forward(x, 2, 1)
    with pytest.raises(ValueError):
        tp.tp_attn_core_backward(torch.zeros(4, 128), x, torch.zeros(4, 128), torch.zeros(2, 4), 2, 1)


@pytest.mark.parametrize("call", [forward, backward])
def test_how_long_a_unit_of_work_may_take(L, call):
    for bad in ({"T": (1 << 26) + 1, "n": 1, "kv": 1}, {"T": (1 << 20) + 1, "n": 64, "kv": 1},
                {"T": 1 << 21, "n": 64, "kv": 1, "window": 1 << 20, "sinks": 1},
                {"T": 1 << 21, "n": 64, "kv": 1, "window": 1 << 20}):
        assert call(L, **bad) == SHAPE and b"2^26" in L.tpce_last_error(), bad
    # not refused for that: a misaligned pointer is what these are turned down for
    room = {"size": 1 << 40} if call is backward else {}
    for fine in ({"T": 1 << 20, "n": 64, "kv": 1}, {"T": 1 << 21, "n": 64, "kv": 1, "window": 4096},
                 {"T": 1 << 27, "n": 1, "kv": 1, "dtype": 1}):
        assert call(L, O=3 * MB + 8, **room, **fine) == ALIGN, fine
    assert call(L, scale=3e38) == INVALID


@pytest.mark.parametrize("call", [forward, backward])
def test_how_long_the_search_for_a_unit_may_take(L, call):
    one = {"n": 1, "kv": 1}
    for bad in ({"b": (1 << 26) + 1, **one}, {"b": 1 << 29, **one}, {"b": (1 << 26) + 1, "scale": -1.0, **one}):
        assert call(L, **bad) == SHAPE and b"2^26" in L.tpce_last_error(), bad
    # not refused for that: a misaligned pointer is what these are turned down for
    for fine in ({"b": 1 << 26, **one}, {"b": 1 << 29, "dtype": 1, **one}, {"b": 1 << 29, "offsets": 0, **one}):
        assert call(L, O=3 * MB + 8, **fine) == ALIGN, fine
