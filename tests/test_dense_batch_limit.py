"""Dense attention bounds the number of sequences on the host (no GPU needed)."""
import ctypes

import pytest

FAKE = ctypes.c_void_p(0x10000)


@pytest.fixture(scope="module")
def s5():
    from block_sparse_gqa_indexer_b200 import build
    build.build()
    from block_sparse_gqa_indexer_b200 import s5 as mod
    return mod


@pytest.mark.parametrize("batch,refused", [((1 << 20) + 1, True), (2 ** 31 - 1, True), (1 << 20, False)])
def test_more_sequences_than_the_kernel_takes(s5, batch, refused):
    """(A batch within the limit gets as far as the next check, the missing workspace.)"""
    b = ctypes.byref(s5.BatchDesc(0x10000, 0x20000, 0x30000, batch, 64, 2, 1, 4000))
    kv = ctypes.byref(s5.KvDesc(0x10000, 0x10000, 8, 64, 4, 192))
    want = s5.S5_ERR_UNSUPPORTED if refused else s5.S5_ERR_WORKSPACE
    assert s5._lib.s5_dense_gqa_attn(kv, b, FAKE, 0.1, FAKE, None, None, 0, None) == want
    assert s5._lib.s5_dense_gqa_attn_fp8kv(kv, b, FAKE, 0.1, 1.0, 1.0, FAKE, None, None, 0, None) == want
