"""The embedding's refusals and workspace sizes, on the CPU: every call here is
turned down by the library's host checks (the pointers are never read)."""

import ctypes

import pytest

P = ctypes.c_void_p
OK = P(1 << 20)
ODD = P((1 << 20) + 8)
INVALID, SHAPE, ALIGN, WORKSPACE = 1, 2, 3, 4


@pytest.fixture(scope="module")
def L():
    from vocab_ce_gb300 import build
    build.build()
    from vocab_ce_gb300._lib import lib
    return lib()


def test_forward_refusals(L):
    def call(T=4, h=64, v_pad=128, v=100, scale=1.0, dtype=0, ids=P(1 << 20), E=P(2 << 20), X=P(3 << 20)):
        return L.tp_embedding_forward(ids, E, T, h, v_pad, v, scale, dtype, X, None)
    assert call(T=0, ids=None, E=None, X=None) == 0
    assert call(T=-1) == SHAPE and call(T=(1 << 28) + 1) == SHAPE
    assert call(h=0) == SHAPE and call(h=60) == SHAPE and call(h=(1 << 20) + 8) == SHAPE
    assert call(v_pad=0, v=0) == SHAPE and call(v=0) == SHAPE and call(v=129) == SHAPE
    assert call(v_pad=(1 << 30) + 1) == SHAPE
    assert call(T=1 << 28, h=1 << 13) == SHAPE and call(v_pad=1 << 28, h=1 << 13) == SHAPE
    assert call(dtype=2) == INVALID and call(dtype=-1) == INVALID
    assert call(scale=float("inf")) == INVALID and call(scale=float("nan")) == INVALID
    for name in ("ids", "E", "X"):
        assert call(**{name: None}) == INVALID and call(**{name: ODD}) == ALIGN
    # X inside what is read
    assert call(X=P(1 << 20)) == INVALID and call(X=P((2 << 20) + 99 * 128)) == INVALID
    assert call(X=P((2 << 20) - 3 * 128)) == INVALID and b"overlap" in L.tpce_last_error()


def test_backward_refusals(L):
    def call(T=4, h=64, v_pad=128, v=100, scale=1.0, dtype=0, add=0, dX=P(1 << 20), ids=P(2 << 20), dE=P(3 << 20),
             ws=P(4 << 20), n=1 << 30):
        return L.tp_embedding_backward(dX, ids, T, h, v_pad, v, scale, dtype, add, dE, ws, n, None)
    assert call(T=0, dX=None, ids=None, dE=None, ws=None, add=1) == 0
    assert call(T=0, dE=None) == INVALID
    assert call(T=-1) == SHAPE and call(h=12) == SHAPE and call(v=0) == SHAPE and call(v=129) == SHAPE
    assert call(dtype=7) == INVALID and call(scale=float("-inf")) == INVALID
    for name in ("dX", "ids", "dE"):
        assert call(**{name: None}) == INVALID and call(**{name: ODD}) == ALIGN
    assert call(ws=ODD) == ALIGN
    need = L.tpce_embedding_workspace_bytes(4, 64, 128)
    assert need > 0 and call(ws=None) == WORKSPACE and call(n=need - 1) == WORKSPACE
    assert str(need) in L.tpce_last_error().decode()
    for bad in ({"dE": P(1 << 20)}, {"dE": P((2 << 20) - 16)}, {"ws": P(1 << 20)}, {"ws": P((3 << 20) + 127 * 128)}):
        assert call(**bad) == INVALID and b"overlap" in L.tpce_last_error(), bad


def test_workspace(L):
    import vocab_ce_gb300 as tp
    need = tp.embedding_workspace_bytes
    assert need(0, 64, 128) == 0 and need(-1, 64, 128) == 0 and need(4, 60, 128) == 0 and need(4, 64, 0) == 0
    for T, h, v in ((1, 8, 1), (16, 64, 100), (17, 64, 100), (16384, 8192, 129024), (1 << 20, 1024, 1 << 20)):
        chunks = -(-T // max(16, -(-T // 1024)))
        sums = 2 * chunks * h * 4 if chunks > 1 else 0
        # the sums, the sorted keys and tokens twice, and at most 256 blocks' counts of 1024 digits
        assert sums + 16 * T <= need(T, h, v) <= sums + 16 * T + 2048 + 256 * 4096, (T, h, v)


def test_without_a_built_binding_or_gpu_nothing_runs_on_the_cpu(L):
    torch = pytest.importorskip("torch")
    import vocab_ce_gb300 as tp
    ids, E = torch.zeros(4, dtype=torch.int32), torch.zeros(8, 64)
    with pytest.raises(ValueError, match="CUDA"):
        tp.tp_embedding_forward(ids, E)
    with pytest.raises(ValueError, match="CUDA"):
        tp.tp_embedding_backward(torch.zeros(4, 64), ids, 8)


def test_workspace_holds_every_part(L):
    import vocab_ce_gb300 as tp
    for T in (1, 8, 9, 16, 17, 999, 2047, 2048, 2049, 4096, 4097, 16_384, 16_385, 65_536, 65_537, 1 << 20):
        for h, v in ((8, 5), (64, 100), (1000, 30_001), (8192, 129_024), (64, 1 << 24)):
            chunk = max(8 if T <= 2048 else 16, -(-T // 1024))
            chunks = -(-T // chunk)
            sums = 2 * chunks * h * 4 if chunks > 1 else 0
            sorted_ids = 4 * (-(-4 * T // 256) * 256)
            # more tokens than one launch sorts: counts of up to 1024 digits by up to 256 blocks
            counts = 256 * 4096 if T > 65_536 else 0
            need = tp.embedding_workspace_bytes(T, h, v)
            assert sorted_ids + sums <= need <= sorted_ids + sums + counts, (T, h, v)
            if counts:
                assert need > sorted_ids + sums
