"""The workspace of the block selection grows with the rows, not with the score matrix."""
import ctypes

import pytest

import block_sparse_attention_tsr_gb300 as tsr


@pytest.fixture(scope="module")
def L():
    tsr.build()
    return tsr.lib()


def size(L, **kw):
    d, n = tsr._SelectDesc(), ctypes.c_size_t(0)
    for k, v in dict(dict(B=1, H=24, d=128, bq=64, bk=64, keep=100), **kw).items():
        setattr(d, k, v)
    assert L.tsr_block_select_workspace(ctypes.byref(d), ctypes.byref(n)) == 0
    return n.value


@pytest.mark.parametrize("bq,bk", [(64, 64), (16, 128), (128, 16)])
def test_linear_in_the_length(L, bq, bk):
    """Means, norms and fragments double with N; where rows outgrow shared memory, one
    strip of 16 rows (whole chunks of 32 blocks and 4 more) for each of 456 CTAs comes in."""
    sizes = [(1 << s, size(L, N=1 << s, bq=bq, bk=bk)) for s in range(17, 25)]
    for (_, a), (n, b) in zip(sizes, sizes[1:]):
        assert b <= 2.01 * a + 456 * 16 * 4 * (n // bk + 36)


def test_linear_in_the_heads(L):
    assert size(L, N=1 << 18, H=48) <= 2 * size(L, N=1 << 18, H=24)


def test_a_million_tokens(L):
    """24 heads of 2^20 tokens: means, norms and fragments 1.2 GB, one strip of scores
    for each resident CTA 0.5 GB (the whole score matrix would be 26 GB)."""
    assert size(L, N=1 << 20) < 2 << 30


def test_too_many_blocks_are_refused_before_the_workspace_is_made(L):
    """2^31 blocks: the query says so, instead of a size that no device holds."""
    d, n = tsr._SelectDesc(), ctypes.c_size_t(0)
    d.B, d.H, d.N, d.d, d.bq, d.bk, d.keep = 1, 1 << 10, 1 << 24, 64, 16, 16, 1
    assert L.tsr_block_select_workspace(ctypes.byref(d), ctypes.byref(n)) == 2
    assert b"2^31" in L.tsr_last_error()
    assert L.tsr_block_select(ctypes.byref(d), 4096, 8192, 12288, 16384, 1 << 62, None) == 2
    d.N = (1 << 24) - 16                                     # 2^31 - 2^11 blocks
    assert L.tsr_block_select_workspace(ctypes.byref(d), ctypes.byref(n)) == 0 and n.value > 0
