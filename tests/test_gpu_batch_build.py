"""A step's batch tables built on the GPU (``s5_build_batch``) against a plain
host construction, and a run of table build, cache append and dense attention."""
import math
import random

import pytest
import torch

pytestmark = pytest.mark.gpu

PAGE = 64


def ceil_pages(n):
    return -(-n // PAGE)


def plain(req_pages, req_ids, ctx, new, free, max_pages, total_q):
    """Host construction: table, cu_q, slots, positions, pages used, requests' pages."""
    req = [row[:] for row in req_pages]
    table, cu, slots, positions, used = [], [0], [], [], 0
    for i, c, n in zip(req_ids, ctx, new):
        row = [-1] * max_pages
        if i >= 0:
            held, need = ceil_pages(c), ceil_pages(c + n)
            for p in range(held):
                row[p] = req[i][p]
            for p in range(held, need):
                row[p] = free[used] if used < len(free) else -1
                req[i][p] = row[p]
                used += 1
            for t in range(c, c + n):
                slots.append(row[t // PAGE] * PAGE + t % PAGE if row[t // PAGE] >= 0 else -1)
                positions.append(t)
        table.append(row)
        cu.append(min(len(slots), total_q))
    return table, cu, slots[:total_q], positions[:total_q], min(used, len(free)), req


class Build:
    def __init__(self, lib, ctx, new, max_pages=None, stride=None, n_reqs=None, req_ids=None, n_free=None, seed=0,
                 total_q=None):
        rng = random.Random(seed)
        self.ctx, self.new = list(ctx), list(new)
        n = len(self.ctx)
        need = max([1] + [ceil_pages(c + m) for c, m in zip(ctx, new)])
        self.max_pages = need if max_pages is None else max_pages
        stride = self.max_pages if stride is None else stride
        n_reqs = n + 3 if n_reqs is None else n_reqs
        self.ids = rng.sample(range(n_reqs), n) if req_ids is None else list(req_ids)
        perm = torch.randperm(n_reqs * stride, generator=torch.Generator().manual_seed(seed))
        self.req = perm.view(n_reqs, stride).tolist()
        taken = sum(ceil_pages(c + m) - ceil_pages(c) for i, c, m in zip(self.ids, ctx, new) if i >= 0)
        n_free = taken + 2 if n_free is None else n_free
        self.free = [n_reqs * stride + x for x in rng.sample(range(n_free + 5), n_free)]
        live = sum(m for i, m in zip(self.ids, new) if i >= 0)
        self.total_q = live if total_q is None else total_q
        i32 = dict(dtype=torch.int32, device="cuda")
        self.d_req, self.d_ids = torch.tensor(self.req, **i32), torch.tensor(self.ids, **i32)
        self.d_new, self.d_free = torch.tensor(self.new, **i32), torch.tensor(self.free, **i32)
        table = torch.full((n, self.max_pages), -9, **i32)
        cu = torch.full((n + 1,), -9, **i32)
        max_len = max([1] + [c + m for c, m in zip(ctx, new)])
        self.batch = lib.Batch(table, torch.tensor(self.ctx, **i32), cu, self.total_q, max([1] + self.new), max_len)
        self.slots, self.pos = torch.full((self.total_q,), -9, **i32), torch.full((self.total_q,), -9, **i32)
        self.used = torch.full((1,), -9, **i32)
        self.ws = torch.zeros(lib.S5_WS_FIXED_BYTES, dtype=torch.uint8, device="cuda")

    def call(self, lib, stream=None):
        lib.s5_build_batch(self.d_req, self.d_ids, self.d_new, self.d_free, self.batch, self.slots, self.pos,
                           self.used, self.ws, stream)

    def run(self, lib, code=0):
        self.call(lib)
        torch.cuda.synchronize()
        got = lib.s5_get_device_error(self.ws)
        assert got[0] == code, got
        return self

    def check(self):
        table, cu, slots, pos, used, req = plain(self.req, self.ids, self.ctx, self.new, self.free, self.max_pages,
                                                 self.total_q)
        assert self.batch.page_table.tolist() == table
        assert self.batch.cu_q.tolist() == cu
        n = cu[-1]
        assert self.slots.tolist() == slots + [-9] * (self.total_q - n)
        assert self.pos.tolist() == pos + [-9] * (self.total_q - n)
        assert self.used.item() == used
        assert self.d_req.tolist() == req
        return self


@pytest.mark.parametrize("max_pages", [None, 8, 9, 12, 131])
@pytest.mark.parametrize("ctx,new", [
    ([0], [0]), ([0], [1]), ([63], [1]), ([64], [1]), ([64, 63, 0, 65, 128], [1, 2, 1, 64, 300]),
    ([5, 0, 500, 0], [0, 0, 0, 0]), ([1, 2, 3], [1, 200, 65]),
])
def test_small(lib, ctx, new, max_pages):
    Build(lib, ctx, new, max_pages=max_pages, stride=None if max_pages is None else max_pages + 3, seed=1).run(lib).check()


@pytest.mark.parametrize("n,hi,new_hi", [(255, 3000, 1), (256, 500, 3), (257, 500, 700), (1023, 300, 2), (1024, 9000, 1),
                                         (1025, 300, 2), (3000, 200, 5)])
def test_large(lib, n, hi, new_hi):
    rng = random.Random(n)
    ctx = [rng.randrange(hi + 1) for _ in range(n)]
    new = [rng.randrange(new_hi + 1) for _ in range(n)]
    ids = rng.sample(range(n + 9), n)
    for s in rng.sample(range(n), n // 10):
        ids[s] = -1
    for stride in (None, 1 + max(ceil_pages(c + m) for c, m in zip(ctx, new))):
        Build(lib, ctx, new, req_ids=ids, n_reqs=n + 9, stride=stride, seed=n).run(lib).check()


def test_empty_sequences_and_rows_behind(lib):
    b = Build(lib, [100, 77, 3, 64], [2, 5, 1, 9], req_ids=[1, -1, 0, -1], total_q=8, seed=2).run(lib).check()
    assert b.slots[3:].tolist() == [-9] * 5


def test_free_list_runs_out(lib):
    b = Build(lib, [64, 10, 128], [65, 1, 1], n_free=2, seed=3).run(lib, code=lib.S5_ERR_DEVICE_BOUNDS)
    assert lib.s5_get_device_error(b.ws)[1] == 2
    b.check()


def test_no_free_pages_and_no_rows(lib):
    Build(lib, [64, 10, 0], [0, 3, 0], n_free=0, seed=7).run(lib).check()
    b = Build(lib, [64, 10], [0, 0], n_free=0, seed=8).run(lib).check()
    assert b.total_q == 0 and b.batch.cu_q.tolist() == [0, 0, 0]


def test_rows_beyond_total_q_are_cut(lib):
    b = Build(lib, [64, 10, 128], [3, 4, 2], total_q=5, seed=4).run(lib, code=lib.S5_ERR_DEVICE_BOUNDS)
    assert lib.s5_get_device_error(b.ws)[1] == 1
    b.check()


@pytest.mark.parametrize("field,value", [("id", -2), ("id", 100), ("ctx", -1), ("new", -3), ("ctx", 2147483647),
                                         ("new", 2147483647), ("ctx", 64 * 9)])
def test_bad_sequences_are_empty(lib, field, value):
    b = Build(lib, [64, 10, 128], [3, 4, 2], max_pages=9, n_reqs=10, seed=5)
    {"id": b.d_ids, "ctx": b.batch.ctx_lens, "new": b.d_new}[field][1] = value
    b.run(lib, code=lib.S5_ERR_DEVICE_BOUNDS)
    assert lib.s5_get_device_error(b.ws)[1] == 1
    b.ids[1] = -1
    b.check()


def test_optional_outputs(lib):
    b = Build(lib, [64, 10], [3, 4], seed=6)
    lib.s5_build_batch(b.d_req, b.d_ids, b.d_new, b.d_free, b.batch, None, None, None, b.ws)
    table, cu, *_ = plain(b.req, b.ids, b.ctx, b.new, b.free, b.max_pages, b.total_q)
    assert b.batch.page_table.tolist() == table and b.batch.cu_q.tolist() == cu


@pytest.mark.parametrize("kv", ["bf16", "fp8"])
def test_decode_steps_build_append_attend(lib, kv):
    """Steps of a server, captured once: tables, append of the new tokens, dense attention over the
    cache, replayed while the requests grow over page edges; the cache is checked by the attention."""
    H, G, D = 64, 4, 192
    g = torch.Generator(device="cuda").manual_seed(20)
    i32 = dict(dtype=torch.int32, device="cuda")
    n, n_reqs, max_pages, steps, scale = 3, 5, 4, 70, 1 / 64
    n_pages = 64
    dt = torch.bfloat16 if kv == "bf16" else torch.uint8
    k_pool, v_pool = (torch.full((n_pages, G, PAGE, D), float("nan") if kv == "bf16" else 0x7F, dtype=dt, device="cuda")
                      for _ in range(2))
    req_pages = torch.full((n_reqs, max_pages), -1, **i32)
    free_all = torch.randperm(n_pages, generator=g, device="cuda").to(torch.int32)
    req_ids, new = torch.tensor([4, 0, 2], **i32), torch.tensor([1, 2, 1], **i32)
    ctx = torch.zeros(n, **i32)
    rows = 4
    batch = lib.Batch(torch.zeros((n, max_pages), **i32), ctx, torch.zeros(n + 1, **i32), rows, 2, 256)
    ws = lib.new_workspace(batch, dense=True)
    slots, pos, used = torch.empty(rows, **i32), torch.empty(rows, **i32), torch.empty(1, **i32)
    free = torch.empty(8, **i32)
    q = torch.empty((rows, H, D), dtype=torch.bfloat16, device="cuda")
    kn, vn = (torch.empty((rows, G, D), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    out, lse = torch.empty_like(q), torch.empty((rows, H), device="cuda")
    sm = 1 / math.sqrt(D)

    def step():
        lib.s5_build_batch(req_pages, req_ids, new, free, batch, slots, pos, used, ws)
        if kv == "bf16":
            lib.s5_append_kv(k_pool, v_pool, None, batch, kn, vn, None, ws)
            lib.s5_dense_gqa_attn(k_pool, v_pool, batch, q, sm, out, lse, ws)
        else:
            lib.s5_append_kv_fp8(k_pool, v_pool, None, batch, kn, vn, None, scale, scale, ws)
            lib.s5_dense_gqa_attn_fp8kv(k_pool, v_pool, batch, q, sm, scale, scale, out, lse, ws)

    graph = torch.cuda.CUDAGraph()
    free.copy_(free_all[:8])
    for x in (q, kn, vn):
        x.zero_()
    keep = req_pages.clone()
    step()  # (warm-up; what it wrote is taken back)
    torch.cuda.synchronize()
    req_pages.copy_(keep)
    with torch.cuda.graph(graph):
        step()
    taken, hist = 0, [([], []) for _ in range(n)]
    for it in range(steps):
        free.copy_(free_all[taken:taken + 8])
        for x in (q, kn, vn):
            x.copy_(torch.randn(x.shape, generator=g, device="cuda").to(torch.bfloat16))
        graph.replay()
        torch.cuda.synchronize()
        taken += int(used)
        assert pos.tolist() == [int(ctx[0]), int(ctx[1]), int(ctx[1]) + 1, int(ctx[2])]
        r = 0
        for s in range(n):
            for j in range(int(new[s])):
                for x, h in zip((kn, vn), hist[s]):
                    y = x[r].double()
                    if kv == "fp8":
                        y = (x[r].float() * (1 / scale)).clamp(-448, 448).to(torch.float8_e4m3fn).double() * scale
                    h.append(y)
                k, v = (torch.stack(h, 1) for h in hist[s])  # [group][token][dim]
                qq = q[r].double().view(G, 16, D)
                sc = torch.einsum("ghd,gtd->ght", qq, k) * sm
                w = torch.softmax(sc, -1)
                want = torch.einsum("ght,gtd->ghd", w, v).reshape(H, D)
                mag = torch.einsum("ght,gtd->ghd", w, v.abs()).reshape(H, D)
                # half a bf16 step of the result and of the weights; scores to 2^-12 (|q.K| sm below 100)
                tol = 2.0 ** -8 * want.abs() + (2.0 ** -8 + 2.0 ** -11) * mag
                assert bool(((out[r].double() - want).abs() <= tol).all()), (it, s, j)
                assert bool(((lse[r].double() - torch.logsumexp(sc, -1).reshape(H)).abs() <= 2.0 ** -11).all())
                r += 1
        ctx += new
    assert lib.s5_get_device_error(ws)[0] == 0
