"""Every entry point refuses a workspace that its kernels' loads and stores could not use (no GPU needed)."""
import ctypes

import pytest

FAKE = ctypes.c_void_p(0x10000)
ROOMY = 1 << 40


@pytest.fixture(scope="module")
def s5():
    from block_sparse_gqa_indexer_b200 import build
    build.build()
    from block_sparse_gqa_indexer_b200 import s5 as mod
    return mod


def _calls(s5, ws, total_q=2, max_q=1):
    """(name, status) of every call that takes a workspace, all else being valid."""
    b = ctypes.byref(s5.BatchDesc(0x10000, 0x20000, 0x30000, 2, 64, total_q, max_q, 4000))
    kv = ctypes.byref(s5.KvDesc(0x10000, 0x10000, 8, 64, 4, 192))
    ix = ctypes.byref(s5.IndexDesc(0x10000, 8, 256))
    req = ctypes.byref(s5.RequestDesc(0x100000, 0x200000, 4, 4, 3))
    lib, w = s5._lib, (ctypes.c_void_p(ws), ROOMY, None)
    index = [lib.s5_index_score_topk, lib.s5_index_score_topk_fp8, lib.s5_index_score_topk_grouped]
    sparse = [lib.s5_sparse_gqa_attn, lib.s5_sparse_gqa_attn_grouped]
    return ([(f.__name__, lambda f=f: f(ix, b, FAKE, 512, FAKE, FAKE, *w)) for f in index] +
            [(f.__name__, lambda f=f: f(kv, b, FAKE, FAKE, FAKE, 512, 0.1, FAKE, None, *w)) for f in sparse] +
            [("sparse_fp8kv", lambda: lib.s5_sparse_gqa_attn_fp8kv(kv, b, FAKE, FAKE, FAKE, 512, 0.1, 1.0, 1.0, FAKE,
                                                                   None, *w)),
             ("swa", lambda: lib.s5_swa_gqa_attn(kv, b, FAKE, 512, 0.1, FAKE, None, *w)),
             ("dense", lambda: lib.s5_dense_gqa_attn(kv, b, FAKE, 0.1, FAKE, None, *w)),
             ("dense_fp8kv", lambda: lib.s5_dense_gqa_attn_fp8kv(kv, b, FAKE, 0.1, 1.0, 1.0, FAKE, None, *w))],
            [("append", lambda: lib.s5_append_kv(kv, None, b, FAKE, FAKE, None, *w)),
             ("append_fp8", lambda: lib.s5_append_kv_fp8(kv, None, b, FAKE, FAKE, None, 1.0, 1.0, *w)),
             ("build_batch", lambda: lib.s5_build_batch(req, FAKE, FAKE, b, FAKE, FAKE, FAKE, *w))])


@pytest.mark.parametrize("off", [1, 2, 4, 8, 12])
@pytest.mark.parametrize("max_q", [1, 8])
def test_unaligned_workspace_is_refused(s5, off, max_q):
    scratch, record_only = _calls(s5, 0x40000 + off, total_q=2 * max_q, max_q=max_q)
    for name, call in scratch:
        assert call() == s5.S5_ERR_INVALID_ARG, name
    if off % 4:
        for name, call in record_only:
            assert call() == s5.S5_ERR_INVALID_ARG, name


def test_nothing_to_do_is_still_fine(s5):
    scratch, record_only = _calls(s5, 0x40001, total_q=0)
    for name, call in scratch + record_only[:2]:
        assert call() == s5.S5_OK, name
