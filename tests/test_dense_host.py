"""Host-side checks of dense attention and of the batch tables: bad arguments
are refused before anything is enqueued (no GPU needed)."""
import ctypes

import pytest

FAKE = ctypes.c_void_p(0x10000)


@pytest.fixture(scope="module")
def s5():
    from block_sparse_gqa_indexer_b200 import build
    build.build()
    from block_sparse_gqa_indexer_b200 import s5 as mod
    return mod


def _batch(s5, **kw):
    d = dict(page_table=0x10000, ctx_lens=0x20000, cu_q=0x30000, batch=2, max_pages=4, total_q=2, max_q=1, max_len=200)
    d.update(kw)
    return s5.BatchDesc(**d)


def _kv(s5, k=0x10000, v=0x10000, n=8, page=64, groups=4, dim=192):
    return s5.KvDesc(k, v, n, page, groups, dim)


def _dense(s5, fp8, kv=None, b=None, q=FAKE, sm=0.1, ks=1.0, vs=1.0, out=FAKE, ws=FAKE, n=1 << 40):
    kv, b = _kv(s5) if kv is None else kv, _batch(s5) if b is None else b
    if fp8:
        return s5._lib.s5_dense_gqa_attn_fp8kv(ctypes.byref(kv), ctypes.byref(b), q, sm, ks, vs, out, None, ws, n, None)
    return s5._lib.s5_dense_gqa_attn(ctypes.byref(kv), ctypes.byref(b), q, sm, out, None, ws, n, None)


@pytest.mark.parametrize("fp8", [False, True])
def test_dense_refusals(s5, fp8):
    bad, uns, wsp = s5.S5_ERR_INVALID_ARG, s5.S5_ERR_UNSUPPORTED, s5.S5_ERR_WORKSPACE
    for b, want in [(dict(batch=0), bad), (dict(max_pages=0), bad), (dict(total_q=-1), bad), (dict(max_q=0), bad),
                    (dict(max_len=257), bad), (dict(page_table=None), bad), (dict(ctx_lens=None), bad),
                    (dict(cu_q=None), bad), (dict(max_len=(1 << 21) + 1, max_pages=1 << 16), uns),
                    (dict(total_q=1 << 25), uns)]:
        assert _dense(s5, fp8, b=_batch(s5, **b)) == want, b
    for kv, want in [(dict(page=32), uns), (dict(groups=8), uns), (dict(dim=128), uns), (dict(n=0), bad),
                     (dict(n=1 << 23), uns), (dict(k=None), bad), (dict(v=0x10008), bad)]:
        assert _dense(s5, fp8, kv=_kv(s5, **kv)) == want, kv
    for kw, want in [(dict(q=None), bad), (dict(out=None), bad), (dict(q=ctypes.c_void_p(0x10008)), bad),
                     (dict(out=ctypes.c_void_p(0x10002)), bad), (dict(sm=float("nan")), bad),
                     (dict(sm=float("inf")), bad), (dict(ws=None), wsp), (dict(n=64), wsp)]:
        assert _dense(s5, fp8, **kw) == want, kw
    assert _dense(s5, fp8, b=_batch(s5, total_q=0), q=None, out=None, n=0) == s5.S5_OK  # nothing enqueued
    if fp8:
        for ks, vs, sm in [(float("nan"), 1.0, 0.1), (1.0, float("inf"), 0.1), (1e38, 1.0, 1e3)]:
            assert _dense(s5, True, sm=sm, ks=ks, vs=vs) == bad


def test_dense_workspace_size(s5):
    n, m = ctypes.c_size_t(0), ctypes.c_size_t(0)
    for kw in (dict(), dict(batch=64, total_q=64, max_pages=2049, max_len=131073),
               dict(batch=1, total_q=500, max_q=500, max_pages=40, max_len=2000)):
        b = _batch(s5, **kw)
        assert s5._lib.s5_workspace_size_dense(ctypes.byref(b), 512, ctypes.byref(n)) == s5.S5_OK
        assert s5._lib.s5_workspace_size(ctypes.byref(b), 512, ctypes.byref(m)) == s5.S5_OK
        assert n.value >= m.value  # covers the other calls too
        for fp8 in (False, True):
            assert _dense(s5, fp8, b=b, n=s5.S5_WS_FIXED_BYTES - 1) == s5.S5_ERR_WORKSPACE
    assert s5._lib.s5_workspace_size_dense(ctypes.byref(b), -1, ctypes.byref(n)) == s5.S5_ERR_INVALID_ARG
    assert s5._lib.s5_workspace_size_dense(ctypes.byref(b), 0, None) == s5.S5_ERR_INVALID_ARG


def _req(s5, pages=0x100000, free=0x200000, n=4, stride=4, n_free=3):
    return s5.RequestDesc(pages, free, n, stride, n_free)


def test_build_batch_refusals(s5):
    f = s5._lib.s5_build_batch
    bad, uns, wsp = s5.S5_ERR_INVALID_ARG, s5.S5_ERR_UNSUPPORTED, s5.S5_ERR_WORKSPACE

    def call(req=None, b=None, ids=FAKE, new=FAKE, ws=FAKE, n=1 << 20):
        return f(ctypes.byref(_req(s5) if req is None else req), ids, new, ctypes.byref(_batch(s5) if b is None else b),
                 FAKE, FAKE, FAKE, ws, n, None)

    for kw, want in [(dict(pages=None), bad), (dict(n=0), bad), (dict(stride=0), bad), (dict(n_free=-1), bad),
                     (dict(free=None), bad), (dict(pages=0x10010), bad), (dict(pages=0xFFF0), bad)]:
        assert call(req=_req(s5, **kw)) == want, kw  # (the last two overlap the page table)
    for kw, want in [(dict(batch=0), bad), (dict(batch=65536), uns), (dict(max_pages=0), bad), (dict(total_q=-1), bad),
                     (dict(max_pages=(1 << 20) + 1, page_table=0x40000000), uns), (dict(page_table=None), bad),
                     (dict(ctx_lens=None), bad), (dict(cu_q=None), bad)]:
        assert call(b=_batch(s5, **kw)) == want, kw
    assert call(ids=None) == bad and call(new=None) == bad
    assert call(ws=None) == wsp and call(n=s5.S5_WS_FIXED_BYTES - 1) == wsp
    assert f(None, FAKE, FAKE, ctypes.byref(_batch(s5)), FAKE, FAKE, FAKE, FAKE, 1 << 20, None) == bad
    assert f(ctypes.byref(_req(s5)), FAKE, FAKE, None, FAKE, FAKE, FAKE, FAKE, 1 << 20, None) == bad


def test_binding_refuses_bad_tensors(s5, monkeypatch):
    """The binding's argument checks, on CPU tensors (device -1 stands for the current device)."""
    import torch
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: -1)
    x, y = torch.zeros(4, dtype=torch.int32), torch.zeros(4, 4, dtype=torch.int32)
    ptrs = s5._ptrs((torch.int32,) * 3, ("a", "b", "c"), x, None, y)
    assert ptrs == [x.data_ptr(), None, y.data_ptr()]
    # a CPU tensor, a wrong type, a strided one, no tensor at all: _need names it
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0)
    for bad in (x, torch.zeros(4), y.t(), 5, [1]):
        with pytest.raises(TypeError, match="b must be a CUDA tensor"):
            s5._ptrs((torch.int32,) * 2, ("a", "b"), None, bad)

    class Elsewhere(torch.Tensor):  # passes for a tensor of another device
        is_cuda = True

        def get_device(self):
            return 3

    t = torch.zeros(4, dtype=torch.int32).as_subclass(Elsewhere)
    with pytest.raises(ValueError, match="a is on cuda:3, the current device is cuda:0"):
        s5._ptrs((torch.int32,), ("a",), t)
