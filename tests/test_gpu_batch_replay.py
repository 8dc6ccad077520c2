"""A full-attention layer's step (tables, cache append, dense attention, lengths and free list moved on)
captured once and replayed without the host looking at anything in between."""
import math

import pytest
import torch

from tests.test_gpu_batch_build import PAGE, plain

pytestmark = pytest.mark.gpu

H, G, D = 64, 4, 192


@pytest.mark.parametrize("kv", ["bf16", "fp8"])
def test_steps_that_only_the_gpu_advances(lib, kv):
    g = torch.Generator(device="cuda").manual_seed(30)
    i32 = dict(dtype=torch.int32, device="cuda")
    n_reqs, max_pages, steps, n_pages, scale = 6, 5, 130, 24, 1 / 64
    ids, new, start = [4, -1, 0, 2], [1, 3, 2, 1], [0, 0, 60, 63]  # (a padded place among them)
    n, rows, sm = len(ids), 4, 1 / math.sqrt(D)
    dt = torch.bfloat16 if kv == "bf16" else torch.uint8
    k_pool, v_pool = (torch.zeros((n_pages, G, PAGE, D), dtype=dt, device="cuda") for _ in range(2))
    order = torch.randperm(n_pages, generator=g, device="cuda").to(torch.int32)
    held, free = order[:2], order[2:].clone()
    req_pages = torch.full((n_reqs, max_pages), -1, **i32)
    req_pages[0, 0], req_pages[2, 0] = held[0], held[1]  # the started requests hold their first page (zeros)
    req0, free0 = req_pages.tolist(), free.tolist()
    req_ids, new_lens, ctx = torch.tensor(ids, **i32), torch.tensor(new, **i32), torch.tensor(start, **i32)
    batch = lib.Batch(torch.zeros((n, max_pages), **i32), ctx, torch.zeros(n + 1, **i32), rows, 3, max_pages * PAGE)
    ws = lib.new_workspace(batch, dense=True)
    slots, pos, used = torch.zeros(rows, **i32), torch.zeros(rows, **i32), torch.zeros(1, **i32)
    place = torch.arange(free.numel(), device="cuda")
    kn, vn, q = (torch.randn((steps, rows, x, D), generator=g, device="cuda").to(torch.bfloat16) for x in (G, G, H))
    outs, lses = torch.zeros((steps, rows, H, D), dtype=torch.bfloat16, device="cuda"), torch.zeros((steps, rows, H), device="cuda")
    logs = torch.full((steps, 2 * rows + n + 2 + n * max_pages), -9, **i32)
    it = torch.zeros(1, dtype=torch.int64, device="cuda")
    out, lse = torch.zeros_like(outs[0]), torch.zeros_like(lses[0])

    def step():
        k1, v1, q1 = kn[it][0], vn[it][0], q[it][0]
        lib.s5_build_batch(req_pages, req_ids, new_lens, free, batch, slots, pos, used, ws)
        if kv == "bf16":
            lib.s5_append_kv(k_pool, v_pool, None, batch, k1, v1, None, ws)
            lib.s5_dense_gqa_attn(k_pool, v_pool, batch, q1, sm, out, lse, ws)
        else:
            lib.s5_append_kv_fp8(k_pool, v_pool, None, batch, k1, v1, None, scale, scale, ws)
            lib.s5_dense_gqa_attn_fp8kv(k_pool, v_pool, batch, q1, sm, scale, scale, out, lse, ws)
        outs.index_copy_(0, it, out[None])
        lses.index_copy_(0, it, lse[None])
        logs.index_copy_(0, it, torch.cat([slots, pos, batch.cu_q, used, batch.page_table.flatten()])[None])
        ctx.add_(torch.where(req_ids >= 0, new_lens, 0))
        # the pages left move to the front of the list, -1 behind them
        at = place + used
        free.copy_(torch.where(at < free.numel(), free[at.clamp_max(free.numel() - 1)], -1))
        it.add_(1)

    state = [x.clone() for x in (req_pages, ctx, free, it, k_pool, v_pool, slots, pos)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()  # (warm-up; what it wrote is taken back)
    torch.cuda.current_stream().wait_stream(side)
    for x, y in zip((req_pages, ctx, free, it, k_pool, v_pool, slots, pos), state):
        x.copy_(y)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for _ in range(steps):
        graph.replay()
    torch.cuda.synchronize()
    assert lib.s5_get_device_error(ws)[0] == 0

    # the same steps on the host
    req, left, lens = req0, free0, list(start)
    live = sum(m for i, m in zip(ids, new) if i >= 0)
    hist = [([torch.zeros(G, D, dtype=torch.float64, device="cuda")] * c,) * 2 for c in start]
    hist = [(list(a), list(b)) for a, b in hist]
    for t in range(steps):
        table, cu, sl, ps, taken, req = plain(req, ids, lens, new, left, max_pages, rows)
        left = left[taken:]
        got = logs[t].tolist()
        assert got[:live] == sl and got[rows:rows + live] == ps, t
        assert got[2 * rows:2 * rows + n + 1] == cu and got[2 * rows + n + 1] == taken, t
        assert got[2 * rows + n + 2:] == [p for row in table for p in row], t
        r = 0
        for s in range(n):
            if ids[s] < 0:
                continue
            for _ in range(new[s]):
                for x, h in zip((kn, vn), hist[s]):
                    y = x[t, r].double()
                    if kv == "fp8":
                        y = (x[t, r].float() * (1 / scale)).clamp(-448, 448).to(torch.float8_e4m3fn).double() * scale
                    h.append(y)
                if t % 16 == 15 or t == steps - 1:
                    k, v = (torch.stack(h, 1) for h in hist[s])  # [group][token][dim]
                    sc = torch.einsum("ghd,gtd->ght", q[t, r].double().view(G, 16, D), k) * sm
                    w = torch.softmax(sc, -1)
                    want = torch.einsum("ght,gtd->ghd", w, v).reshape(H, D)
                    mag = torch.einsum("ght,gtd->ghd", w, v.abs()).reshape(H, D)
                    # half a bf16 step of the result; weights in two bf16 terms, or (three rows a tile's
                    # bound of max_q = 3) three terms of 3 bits; scores to 2^-12 (|q.K| sm below 100), twice
                    tol = 2.0 ** -8 * want.abs() + ((2.0 ** -15 if kv == "bf16" else 2.0 ** -9) + 2.0 ** -11) * mag
                    assert bool(((outs[t, r].double() - want).abs() <= tol).all()), (t, s)
                    assert bool(((lses[t, r].double() - torch.logsumexp(sc, -1).reshape(H)).abs() <= 2.0 ** -11).all())
                r += 1
        lens = [c + (m if i >= 0 else 0) for c, m, i in zip(lens, new, ids)]
    assert free.tolist() == left + [-1] * (len(free0) - len(left)) and ctx.tolist() == lens
