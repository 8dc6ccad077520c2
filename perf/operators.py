"""Workloads of the two operators around a paged key-value cache: dense attention of new tokens over it, and the
page tables, row offsets and slots that a step's batch needs, built on the GPU from the requests' lengths.

A module-level ``own`` chooses what ``run`` does: False computes the operators from elementary torch operations in
32 bits, True makes the calls that a user of this package makes.
"""
import math

import torch

own = False

HEADS, GROUPS, DIM, PAGE = 64, 4, 192, 64
PER_GROUP = HEADS // GROUPS
SM_SCALE = 1.0 / math.sqrt(DIM)
FP8_SCALE = 1.0 / 64.0  # a one-byte cache of values of about 1: codes of about 64


def listed():
    return [
        # a step's tables for a few chats with short histories: launch latency
        {"name": "tables_8_short", "op": "tables", "batch": 8, "pad": 0, "ctx_lo": 1, "ctx_hi": 4095, "new_hi": 1},
        # a decode step of 64 requests with long histories
        {"name": "tables_64_long", "op": "tables", "batch": 64, "pad": 0, "ctx_lo": 100000, "ctx_hi": 131072, "new_hi": 1},
        # an odd number of requests verifying a few draft tokens each, in a batch padded to a fixed size
        {"name": "tables_333_verify", "op": "tables", "batch": 333, "pad": 19, "ctx_lo": 0, "ctx_hi": 20000, "new_hi": 5},
        # prefill chunks of 16 requests: thousands of slots
        {"name": "tables_16_chunks", "op": "tables", "batch": 16, "pad": 0, "ctx_lo": 0, "ctx_hi": 32768, "new_hi": 2048},
        # the largest step: a thousand requests of up to 131,072 tokens
        {"name": "tables_1024_long", "op": "tables", "batch": 1024, "pad": 0, "ctx_lo": 1, "ctx_hi": 131072, "new_hi": 1},
        # one chat with a short history: latency of the smallest call
        {"name": "dense_1_short", "op": "dense", "kv": "bf16", "batch": 1, "ctx_lo": 1000, "ctx_hi": 1000, "nq": 1},
        # one request with a long history: its cache has to be split over the whole GPU
        {"name": "dense_1_long", "op": "dense", "kv": "bf16", "batch": 1, "ctx_lo": 131071, "ctx_hi": 131071, "nq": 1},
        # an ordinary decode batch: ragged histories
        {"name": "dense_64_ragged", "op": "dense", "kv": "bf16", "batch": 64, "ctx_lo": 1, "ctx_hi": 16383, "nq": 1},
        # draft tokens being verified: up to 4 rows share a sequence's cache
        {"name": "dense_16_verify", "op": "dense", "kv": "bf16", "batch": 16, "ctx_lo": 20000, "ctx_hi": 32768, "nq": 4},
        # the largest: 32 requests with 131,072 cached tokens each
        {"name": "dense_32_long", "op": "dense", "kv": "bf16", "batch": 32, "ctx_lo": 131072, "ctx_hi": 131072, "nq": 1},
        # one-byte cache, small odd batch
        {"name": "dense8_7_medium", "op": "dense", "kv": "fp8", "batch": 7, "ctx_lo": 500, "ctx_hi": 8191, "nq": 1},
        # one-byte cache, a full decode batch
        {"name": "dense8_64_long", "op": "dense", "kv": "fp8", "batch": 64, "ctx_lo": 30000, "ctx_hi": 65536, "nq": 1},
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    if rng.random() < 0.4:
        batch = _log(rng, 1, 1024)
        ctx_hi = _log(rng, 64, 131072)
        new_hi = rng.choice([1, 1, 2, 5, 8, min(2048, max(1, 32768 // batch))])
        return {"op": "tables", "batch": batch, "pad": rng.randrange(0, batch // 8 + 1),
                "ctx_lo": rng.choice([0, 1, ctx_hi // 2]), "ctx_hi": ctx_hi, "new_hi": new_hi}
    batch = _log(rng, 1, 64)
    nq = rng.choice([1, 1, 1, 2, 3, 4, 5, 8])
    ctx_hi = _log(rng, 16, min(131072, 32 * 131072 // (batch * nq)))
    return {"op": "dense", "kv": rng.choice(["bf16", "fp8"]), "batch": batch,
            "ctx_lo": rng.choice([0, ctx_hi // 2, ctx_hi]), "ctx_hi": ctx_hi, "nq": nq}


# ---------------------------------------------------------------- inputs


def _new_tokens(case, n_max):
    """New tokens of the batch's sequences, in some order: 1 to n_max, their sum the same for every seed."""
    live = case["batch"] - case.get("pad", 0)
    return torch.randint(1, n_max + 1, (live,), generator=torch.Generator().manual_seed(13))


def _lengths(case, n_max, seed):
    """Cached and new tokens of each sequence, as host lists (a scheduler knows them)."""
    g = torch.Generator().manual_seed(seed * 7919 + 13)
    new = _new_tokens(case, n_max)
    ctx = torch.randint(case["ctx_lo"], case["ctx_hi"] + 1, (new.numel(),), generator=g)
    return ctx.tolist(), new[torch.randperm(new.numel(), generator=g)].tolist()


def _lengths_work(case, n_max):
    """Lengths for counting work: (expected cached tokens, new tokens) over the batch."""
    new = _new_tokens(case, n_max)
    return new.numel() * (case["ctx_lo"] + case["ctx_hi"]) / 2, int(new.sum())


def _pages(tokens):
    return -(-tokens // PAGE)


def prepare(case, seed):
    return _prepare_tables(case, seed) if case["op"] == "tables" else _prepare_dense(case, seed)


def _prepare_tables(case, seed):
    ctx, new = _lengths(case, case["new_hi"], seed)
    batch, live = case["batch"], len(ctx)
    g = torch.Generator(device="cuda").manual_seed(seed)
    max_pages = _pages(case["ctx_hi"] + case["new_hi"])
    n_reqs = 2 * batch  # requests that the server holds; a step runs some of them
    perm = torch.randperm(n_reqs * max_pages, generator=g, device="cuda", dtype=torch.int64).to(torch.int32)
    req_ids = torch.full((batch,), -1, dtype=torch.int32, device="cuda")
    req_ids[:live] = torch.randperm(n_reqs, generator=g, device="cuda")[:live].to(torch.int32)
    i32 = dict(dtype=torch.int32, device="cuda")
    ctx_lens = torch.tensor(ctx + [0] * (batch - live), **i32)
    new_lens = torch.tensor(new + [0] * (batch - live), **i32)
    n_new = sum(_pages(c + n) - _pages(c) for c, n in zip(ctx, new))
    state = {"op": "tables", "req_pages": perm.view(n_reqs, max_pages), "req_ids": req_ids, "ctx_lens": ctx_lens,
             "new_lens": new_lens, "rows": sum(new), "max_pages": max_pages,
             # pages that no request holds, in the order in which they are taken
             "free_pages": n_reqs * max_pages + torch.randperm(n_new + 64, generator=g, device="cuda").to(torch.int32)}
    if own:
        from block_sparse_gqa_indexer_b200 import s5
        rows = state["rows"]
        table = torch.empty((batch, max_pages), **i32)
        cu_q = torch.empty((batch + 1,), **i32)
        state["batch"] = s5.Batch(table, ctx_lens, cu_q, rows, max(new), max(c + n for c, n in zip(ctx, new)))
        state["slots"], state["positions"] = torch.empty((rows,), **i32), torch.empty((rows,), **i32)
        state["used"] = torch.empty((1,), **i32)
        state["ws"] = s5.new_workspace(state["batch"])
        state["call"] = s5.s5_build_batch
    return state


def _pool(pages, kv, g):
    """K or V pool [pages][group][token][dim]: values of about 1, in bf16 or as one-byte E4M3 codes."""
    pool = torch.empty((pages, GROUPS, PAGE, DIM), dtype=torch.bfloat16 if kv == "bf16" else torch.uint8, device="cuda")
    step = 8192  # in pieces, so that the drawing needs little memory beside the pool
    for i in range(0, pages, step):
        x = torch.randn((min(step, pages - i), GROUPS, PAGE, DIM), dtype=torch.bfloat16, generator=g, device="cuda")
        pool[i:i + step] = x if kv == "bf16" else (x / FP8_SCALE).clamp_(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
    return pool


def _prepare_dense(case, seed):
    ctx, new = _lengths(case, case["nq"], seed)
    batch, rows, g = case["batch"], sum(new), torch.Generator(device="cuda").manual_seed(seed)
    need = [_pages(c + n) for c, n in zip(ctx, new)]
    k_pool, v_pool = _pool(sum(need), case["kv"], g), _pool(sum(need), case["kv"], g)
    # every page somewhere in the pool; entries behind a sequence's last page hold some other page
    order = torch.randperm(sum(need), generator=g, device="cuda").to(torch.int32)
    first = torch.tensor([sum(need[:s]) for s in range(batch)], device="cuda")
    col = torch.arange(max(need), device="cuda")
    table = order[torch.clamp(first[:, None] + col, max=sum(need) - 1)].contiguous()
    cu = [sum(new[:s]) for s in range(batch + 1)]
    i32 = dict(dtype=torch.int32, device="cuda")
    state = {"op": "dense", "kv": case["kv"], "k_pool": k_pool, "v_pool": v_pool, "table": table,
             "ctx_lens": torch.tensor(ctx, **i32), "cu_q": torch.tensor(cu, **i32), "max_q": max(new), "rows": rows,
             "q": torch.randn((rows, HEADS, DIM), generator=g, device="cuda").to(torch.bfloat16)}
    if own:
        from block_sparse_gqa_indexer_b200 import s5
        state["batch"] = s5.Batch(table, state["ctx_lens"], state["cu_q"], rows, max(new),
                                  max(c + n for c, n in zip(ctx, new)))
        state["ws"] = s5.new_workspace(state["batch"], dense=True)
        state["out"] = torch.empty((rows, HEADS, DIM), dtype=torch.bfloat16, device="cuda")
        state["lse"] = torch.empty((rows, HEADS), dtype=torch.float32, device="cuda")
        state["call"] = s5.s5_dense_gqa_attn if case["kv"] == "bf16" else s5.s5_dense_gqa_attn_fp8kv
    return state


# ---------------------------------------------------------------- one pass


def run(state):
    if own:
        return _run_own(state)
    return _tables(state) if state["op"] == "tables" else _dense(state)


def _run_own(st):
    if st["op"] == "tables":
        st["call"](st["req_pages"], st["req_ids"], st["new_lens"], st["free_pages"], st["batch"], st["slots"],
                   st["positions"], st["used"], st["ws"])
        return {"table": st["batch"].page_table, "cu_q": st["batch"].cu_q, "slots": st["slots"],
                "positions": st["positions"], "used": st["used"], "req_pages": st["req_pages"]}
    if st["kv"] == "bf16":
        st["call"](st["k_pool"], st["v_pool"], st["batch"], st["q"], SM_SCALE, st["out"], st["lse"], st["ws"])
    else:
        st["call"](st["k_pool"], st["v_pool"], st["batch"], st["q"], SM_SCALE, FP8_SCALE, FP8_SCALE, st["out"],
                   st["lse"], st["ws"])
    return {"out": st["out"], "lse": st["lse"]}


def _tables(st):
    """held / need: pages before and after the step; a sequence's new pages follow those of the sequences before it."""
    live = st["req_ids"] >= 0
    ids = torch.clamp(st["req_ids"], min=0).long()
    ctx, new = st["ctx_lens"].long() * live, st["new_lens"].long() * live
    held, need = (ctx + PAGE - 1) // PAGE, (ctx + new + PAGE - 1) // PAGE
    taken = torch.cumsum(need - held, 0)
    before = (taken - (need - held))[:, None]
    col = torch.arange(st["max_pages"], device="cuda")[None, :]
    fresh = (col >= held[:, None]) & (col < need[:, None])
    free = st["free_pages"][torch.clamp(before + col - held[:, None], 0, st["free_pages"].numel() - 1)]
    old = st["req_pages"][ids]
    table = torch.where(fresh, free, torch.where(col < held[:, None], old, -1))
    at, page = torch.nonzero(fresh, as_tuple=True)
    st["req_pages"][ids[at], page] = table[at, page]
    cu_q = torch.zeros(new.numel() + 1, dtype=torch.int64, device="cuda")
    cu_q[1:] = torch.cumsum(new, 0)
    row = torch.arange(st["rows"], device="cuda")
    seq = torch.searchsorted(cu_q, row, right=True) - 1
    pos = ctx[seq] + row - cu_q[seq]
    slots = table[seq, pos // PAGE] * PAGE + pos % PAGE
    return {"table": table, "cu_q": cu_q.to(torch.int32), "slots": slots.to(torch.int32),
            "positions": pos.to(torch.int32), "used": taken[-1:].to(torch.int32), "req_pages": st["req_pages"]}


def _values(pool, table, kv):
    """The cache of every sequence as fp32 [sequence][group][token][dim]."""
    x = pool[table.long()]
    x = x.float() if kv == "bf16" else x.view(torch.float8_e4m3fn).float() * FP8_SCALE
    b, p = table.shape
    return x.permute(0, 2, 1, 3, 4).reshape(b, GROUPS, p * PAGE, DIM)


def _dense(st):
    cu, ctx, n = st["cu_q"].long(), st["ctx_lens"].long(), st["max_q"]
    batch = ctx.numel()
    # rows padded to the longest sequence's: [sequence][row]
    j = torch.arange(n, device="cuda")[None, :]
    has = j < (cu[1:] - cu[:-1])[:, None]
    row = torch.where(has, cu[:-1, None] + j, 0)
    pos = ctx[:, None] + j
    q = st["q"][row].float().view(batch, n, GROUPS, PER_GROUP, DIM).permute(0, 2, 1, 3, 4)
    q = q.reshape(batch, GROUPS, n * PER_GROUP, DIM)
    s = torch.matmul(q, _values(st["k_pool"], st["table"], st["kv"]).transpose(2, 3)) * SM_SCALE
    tok = torch.arange(s.shape[-1], device="cuda")
    seen = tok[None, None, :] <= pos[:, :, None]
    s = s.view(batch, GROUPS, n, PER_GROUP, -1).masked_fill_(~seen[:, None, :, None, :], float("-inf"))
    top = s.amax(-1, keepdim=True)
    p = torch.exp(s - top)
    total = p.sum(-1, keepdim=True)
    lse = (top + torch.log(total)).squeeze(-1)
    del s
    o = torch.matmul(p.view(batch, GROUPS, n * PER_GROUP, -1), _values(st["v_pool"], st["table"], st["kv"]))
    o = o.view(batch, GROUPS, n, PER_GROUP, DIM) / total
    at, jj = torch.nonzero(has, as_tuple=True)  # rows in order
    return {"out": o.permute(0, 2, 1, 3, 4)[at, jj].reshape(-1, HEADS, DIM).to(torch.bfloat16),
            "lse": lse.permute(0, 2, 1, 3)[at, jj].reshape(-1, HEADS)}


# ---------------------------------------------------------------- what a pass cannot do without


def work(case):
    if case["op"] == "tables":
        ctx, new = _lengths_work(case, case["new_hi"])
        max_pages = _pages(case["ctx_hi"] + case["new_hi"])
        held, fresh = ctx / PAGE, new / PAGE
        # lengths and ids in; held and fresh pages in; the table, row offsets, slots, positions and the requests' new
        # pages out
        return {"bytes": 4 * (4 * case["batch"] + held + 2 * fresh + case["batch"] * max_pages + 2 * new), "flops": 0}
    ctx, new = _lengths_work(case, case["nq"])
    width = 2 if case["kv"] == "bf16" else 1
    mean = ctx / case["batch"]
    return {"bytes": (ctx + new) * 2 * GROUPS * DIM * width + new * HEADS * (2 * 2 * DIM + 4),
            "flops": 4 * HEADS * DIM * new * (mean + 1)}


# ---------------------------------------------------------------- the definition in 64 bits


def exact(case, seed):
    if case["op"] == "tables":
        return None  # whole numbers: they have to be equal
    st = _prepare_dense(case, seed)
    cu, ctx = st["cu_q"].tolist(), st["ctx_lens"].tolist()

    def cached(pool, s, length):
        x = pool[st["table"][s, :_pages(length)].long()].transpose(0, 1).reshape(GROUPS, -1, DIM)[:, :length]
        return x.double() if case["kv"] == "bf16" else x.contiguous().view(torch.float8_e4m3fn).double() * FP8_SCALE

    outs, lses = [], []
    for s in range(case["batch"]):
        k, v = (cached(st[p], s, ctx[s] + cu[s + 1] - cu[s]) for p in ("k_pool", "v_pool"))
        for r in range(cu[s], cu[s + 1]):
            length = ctx[s] + r - cu[s] + 1
            q = st["q"][r].double().view(GROUPS, PER_GROUP, DIM)
            scores = torch.einsum("ghd,gtd->ght", q, k[:, :length]) / math.sqrt(DIM)
            lse = torch.logsumexp(scores, -1)
            outs.append(torch.einsum("ght,gtd->ghd", torch.exp(scores - lse[..., None]), v[:, :length]).reshape(HEADS, DIM))
            lses.append(lse.reshape(HEADS))
    return {"out": torch.stack(outs), "lse": torch.stack(lses)}
