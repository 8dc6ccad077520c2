"""Dense attention over the whole paged cache (bf16 and one-byte KV) on the GPU
against the formula in 64 bits.

Tolerances, derived from the roundings of the computation.  With A = sum_j w_j |V_j|
(the softmax-weighted magnitude of the values) and B = sm_scale * max_j sum_d |q_d K_jd|:
  output rounding        half a bf16 step:               2^-8 |out|
  weights                rounded to bf16 (bf16 KV):      2^-8 A
                         one byte, up to 2 rows a sequence: to 11 bits, 2^-11 A (max_q <= 2); else
                         three terms of 3 bits.  Two terms cut toward zero leave less than
                         2^-5 of the weight's power of two, which the third rounds to 3 of
                         its bits: off by at most 2^-5 / 2 / 2^3 = 2^-9:  2^-9 A
                         one byte, all rows: weights are multiples of 2^-16 where the largest is
                         at least 2^12, cut toward zero:  2^-28 sum_j |V_j|
  scores                 192 fp32 products and the scale: every weight off by
                         a factor of at most 1 +- 200 * 2^-24 B + 2^-20 (exp2 of
                         a scaled, shifted score), in the sum and the quotient: twice that, times A
  long sums              n additions in fp32: 2^-24 n A at most; pieces of at
                         most n / 8 are added, then joined:  2^-27 n A + 2^-20 A
One byte: q is held to 2^-21 of the largest magnitude Q of a group's heads in the rows computed
together, so scores are off by another sm_scale * 2^-22 Q max_j sum_d |K_jd|.
The lse adds the score error, 2^-20 and 2^-27 n, and its own rounding 2^-23 |lse|.
"""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu

H, G, D, PAGE = 64, 4, 192, 64
SM = 1.0 / math.sqrt(D)


def pages(n):
    return -(-n // PAGE)


class Case:
    """A batch over a shuffled pool; entries behind a sequence's pages are -1."""

    def __init__(self, ctx, nq, kv="bf16", seed=0, extra_pages=0, pad_rows=0, k_scale=1.0, v_scale=1.0, sm=SM,
                 max_len=None):
        g = torch.Generator(device="cuda").manual_seed(seed + 1)
        self.ctx, self.nq, self.kv, self.sm = list(ctx), list(nq), kv, sm
        self.k_scale, self.v_scale = (k_scale, v_scale) if kv == "fp8" else (1.0, 1.0)
        need = [pages(c + n) for c, n in zip(ctx, nq)]
        total = sum(need) + 3
        self.order = torch.randperm(total, generator=g, device="cuda").to(torch.int32)
        self.table = torch.full((len(ctx), max(need) + extra_pages), -1, dtype=torch.int32, device="cuda")
        first = 0
        for s, n in enumerate(need):
            self.table[s, :n] = self.order[first:first + n]
            first += n
        x = [torch.randn((total, G, PAGE, D), generator=g, device="cuda") for _ in range(2)]
        if kv == "bf16":
            self.k, self.v = (y.to(torch.bfloat16) for y in x)
        else:
            self.k, self.v = ((y / sc).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
                              for y, sc in zip(x, (k_scale, v_scale)))
        self.cu = [0]
        for n in nq:
            self.cu.append(self.cu[-1] + n)
        self.rows, self.total_q = self.cu[-1], self.cu[-1] + pad_rows
        self.q = torch.randn((self.total_q, H, D), generator=g, device="cuda").to(torch.bfloat16)
        self.max_len = max(c + n for c, n in zip(ctx, nq)) if max_len is None else max_len
        self.max_q = max(1, *nq)

    def make(self, lib):
        i32 = dict(dtype=torch.int32, device="cuda")
        self.batch = lib.Batch(self.table, torch.tensor(self.ctx, **i32), torch.tensor(self.cu, **i32), self.total_q,
                               self.max_q, self.max_len)
        self.ws = lib.new_workspace(self.batch, dense=True)
        self.out = torch.full((self.total_q, H, D), 7.0, dtype=torch.bfloat16, device="cuda")
        self.lse = torch.full((self.total_q, H), 7.0, dtype=torch.float32, device="cuda")
        return self

    def call(self, lib, stream=None, lse=True):
        l = self.lse if lse else None
        if self.kv == "bf16":
            lib.s5_dense_gqa_attn(self.k, self.v, self.batch, self.q, self.sm, self.out, l, self.ws, stream)
        else:
            lib.s5_dense_gqa_attn_fp8kv(self.k, self.v, self.batch, self.q, self.sm, self.k_scale, self.v_scale,
                                        self.out, l, self.ws, stream)

    def run(self, lib, code=0):
        self.make(lib)
        self.call(lib)
        torch.cuda.synchronize()
        got, info = lib.s5_get_device_error(self.ws)
        assert got == code, (lib.s5_status_string(got), info)
        # the partition counters are zero again
        assert int(self.ws[256:lib.S5_WS_FIXED_BYTES].long().sum()) == 0
        return self

    def cached(self, pool, scale, s, n):
        x = pool[self.table[s, :pages(n)].long()].transpose(0, 1).reshape(G, -1, D)[:, :n].contiguous()
        return x.double() if self.kv == "bf16" else x.view(torch.float8_e4m3fn).double() * scale

    def expect(self, s, skip_pages=()):
        """(out, lse, tolerance of out, tolerance of lse) of sequence s's rows, in 64 bits."""
        lo, hi = self.cu[s], self.cu[s + 1]
        n = self.ctx[s] + hi - lo
        k, v = self.cached(self.k, self.k_scale, s, n), self.cached(self.v, self.v_scale, s, n)
        pos = self.ctx[s] + torch.arange(hi - lo, device="cuda")
        tok = torch.arange(n, device="cuda")
        seen = tok[None] <= pos[:, None]
        for p in skip_pages:
            seen &= (tok // PAGE != p)[None]
        # values no row sees may be anything; ones that some rows do not see are masked per row below
        any_seen = seen.any(0)
        k, v = torch.where(any_seen[None, :, None], k, 0.0), torch.where(any_seen[None, :, None], v, 0.0)
        q = self.q[lo:hi].double().view(hi - lo, G, H // G, D)
        sc = torch.einsum("rghd,gtd->rght", q, k) * self.sm
        mag = torch.einsum("rghd,gtd->rght", q.abs(), k.abs()) * abs(self.sm)
        m = seen[:, None, None, :]
        sc = sc.masked_fill(~m, float("-inf"))
        lse = torch.logsumexp(sc, -1)
        w = torch.where(m, torch.exp(sc - torch.where(lse == float("-inf"), 0.0, lse)[..., None]), 0.0)
        if bool(torch.isfinite(v).all()):
            out, a = torch.einsum("rght,gtd->rghd", w, v), torch.einsum("rght,gtd->rghd", w, v.abs())
        else:  # 0 * NaN must not count where a row does not see the token
            term = torch.where(m[..., None], w[..., None] * v[None, :, None], 0.0)
            out, a = term.sum(3), term.abs().sum(3)
        b = mag.masked_fill(~m, 0.0).amax(-1)
        score = 200 * 2.0 ** -24 * b + 2.0 ** -20
        if self.kv == "fp8":
            qmax = torch.where(torch.isfinite(q), q.abs(), 0.0).amax((0, 2, 3))
            score = score + (2.0 ** -22 * abs(self.sm) * qmax * k.abs().sum(-1).amax(-1))[None, :, None]
        weight = 2.0 ** -8 if self.kv == "bf16" else 2.0 ** -11 if self.max_q <= 2 else 2.0 ** -9
        tol = 2.0 ** -8 * out.abs() + (weight + 2 * score + 2.0 ** -27 * n + 2.0 ** -20)[..., None] * a + 1e-30
        if self.kv == "fp8":
            tol = tol + 2.0 ** -28 * v.abs().nan_to_num(0, 0, 0).sum(1)[None, :, None]
        tol_lse = score + 2.0 ** -20 + 2.0 ** -27 * n + 2.0 ** -23 * lse.abs()
        r = hi - lo
        return out.reshape(r, H, D), lse.reshape(r, H), tol.reshape(r, H, D), tol_lse.reshape(r, H)

    def check(self, seqs=None, skip=None):
        for s in range(len(self.ctx)) if seqs is None else seqs:
            lo, hi = self.cu[s], self.cu[s + 1]
            if hi == lo:
                continue
            out, lse, tol, tol_lse = self.expect(s, (skip or {}).get(s, ()))
            got, got_lse = self.out[lo:hi].double(), self.lse[lo:hi].double()
            assert torch.isfinite(got).all() and torch.isfinite(got_lse).all(), s
            over = ((got - out).abs() / tol).max().item()
            over_lse = ((got_lse - lse).abs() / tol_lse).max().item()
            assert over <= 1 and over_lse <= 1, (s, over, over_lse)
        return self


BATCHES = {
    "one_token": ([0], [1]),
    "two": ([1], [1]),
    "page_edges": ([62, 63, 64, 65, 127, 128], [1] * 6),
    "short_1000": ([1000], [1]),
    "verify": ([0, 1, 61, 63, 64, 200], [8, 5, 4, 3, 2, 1]),
    "verify_3": ([700, 5], [3, 3]),
    "verify_4": ([64, 500, 3], [4, 4, 2]),
    "rows_9_17": ([10, 300], [9, 17]),
    "chunk": ([130], [70]),
    "holes": ([5, 70, 0, 64], [0, 1, 0, 2]),
    "ragged": ([3000, 17, 0, 900, 8000, 63], [1] * 6),
    "ragged_verify": ([3000, 17, 0, 900, 5000, 63], [2, 1, 7, 4, 1, 8]),
    "many_short": ([(37 * i) % 200 for i in range(333)], [1 + i % 3 for i in range(333)]),
    "many_empty": ([64] * 1500, [1 if i % 7 == 0 else 0 for i in range(1500)]),
    "long": ([70000], [1]),
    "long_verify": ([40000, 20001], [5, 1]),
}


@pytest.mark.parametrize("kv", ["bf16", "fp8"])
@pytest.mark.parametrize("name", list(BATCHES))
def test_against_formula(lib, name, kv):
    ctx, nq = BATCHES[name]
    Case(ctx, nq, kv, seed=len(name), extra_pages=len(name) % 3, k_scale=0.013, v_scale=0.02).run(lib).check()


@pytest.mark.parametrize("kv", ["bf16", "fp8"])
@pytest.mark.parametrize("name", [n for n, (ctx, nq) in BATCHES.items() if max(c + q for c, q in zip(ctx, nq)) <= 768])
def test_short_sequences_in_a_batch_made_for_long_ones(lib, name, kv):
    """max_len bounds the lengths from far above: tiles may be split over CTAs."""
    ctx, nq = BATCHES[name]
    need = max(pages(c + q) for c, q in zip(ctx, nq))
    c = Case(ctx, nq, kv, seed=30 + len(name), extra_pages=40, k_scale=1 / 64, v_scale=1 / 64, max_len=(need + 40) * PAGE)
    c.run(lib).check()
    wide = c.out.clone()
    d = Case(ctx, nq, kv, seed=30 + len(name), extra_pages=40, k_scale=1 / 64, v_scale=1 / 64).run(lib).check()
    for s in range(len(ctx)):  # the same answers, however the work is divided
        if nq[s]:
            _, _, tol, _ = d.expect(s)
            assert bool(((d.out - wide)[d.cu[s]:d.cu[s + 1]].double().abs() <= 2 * tol).all())


@pytest.mark.parametrize("kv", ["bf16", "fp8"])
def test_without_lse_and_repeatable(lib, kv):
    c = Case([5000, 100, 64], [1, 2, 8], kv, seed=3, k_scale=1 / 64, v_scale=1 / 64).run(lib).check()
    out, lse = c.out.clone(), c.lse.clone()
    c.lse.fill_(7.0)
    for _ in range(5):
        c.out.fill_(9.0)
        c.call(lib, lse=False)
        assert torch.equal(c.out, out)
    assert bool((c.lse == 7.0).all())
    c.call(lib)
    assert torch.equal(c.lse, lse) and torch.equal(c.out, out)


@pytest.mark.parametrize("kv", ["bf16", "fp8"])
@pytest.mark.parametrize("hi,nq", [(300, 1), (700, 8), (4000, 1), (2500, 4)])
def test_ragged_batches_repeat_bit_for_bit(lib, kv, hi, nq):
    """Many sequences per CTA, runs of one chunk among them: right, and the same every time."""
    g = torch.Generator().manual_seed(hi)
    n = 150
    ctx = torch.randint(0, hi, (n,), generator=g).tolist()
    new = torch.randint(1, nq + 1, (n,), generator=g).tolist()
    c = Case(ctx, new, kv, seed=hi + nq, k_scale=1 / 64, v_scale=1 / 64).run(lib).check()
    out, lse = c.out.clone(), c.lse.clone()
    for _ in range(100):
        c.out.fill_(9.0)
        c.call(lib)
        assert torch.equal(c.out, out) and torch.equal(c.lse, lse)


@pytest.mark.parametrize("kv", ["bf16", "fp8"])
def test_rows_behind_the_batch_stay(lib, kv):
    c = Case([500, 3], [2, 1], kv, seed=4, pad_rows=6, k_scale=1 / 64, v_scale=1 / 64).run(lib).check()
    assert bool((c.out[3:] == 7.0).all()) and bool((c.lse[3:] == 7.0).all())


def test_a_padded_batch_without_a_sequence(lib):
    """Rows, but no sequence has new tokens: nothing is written."""
    c = Case([500, 0, 64], [0, 0, 0], seed=23, pad_rows=5, max_len=600, extra_pages=3).run(lib)
    assert bool((c.out == 7.0).all()) and bool((c.lse == 7.0).all())


@pytest.mark.parametrize("kv", ["bf16", "fp8"])
@pytest.mark.parametrize("ctx,nq", [([70, 0, 63, 64, 200], [1, 1, 1, 1, 1]), ([60, 126, 3, 0], [8, 4, 3, 2])])
def test_masked_places_hold_nan_and_infinity(lib, kv, ctx, nq):
    """Slots behind the last position: NaN; rows of a verify batch do not see the later rows' tokens."""
    c = Case(ctx, nq, kv, seed=5, k_scale=1 / 64, v_scale=1 / 64)
    nan = float("nan") if kv == "bf16" else 0x7F
    bad = float("inf") if kv == "bf16" else 0xFF
    for s in range(len(ctx)):
        n = ctx[s] + nq[s]
        page = int(c.table[s, pages(n) - 1])
        if n % PAGE:
            c.k[page, :, n % PAGE:] = nan
            c.v[page, :, n % PAGE:] = nan
            c.v[page, :, -1] = bad
    # unused pages hold NaN as well
    c.k[c.order[-3:].long()] = nan
    c.v[c.order[-3:].long()] = nan
    c.run(lib).check()
    # now the LAST row's own token is NaN: the earlier rows keep their results bit for bit
    out, lse = c.out.clone(), c.lse.clone()
    for s in range(len(ctx)):
        t = ctx[s] + nq[s] - 1
        page = int(c.table[s, t // PAGE])
        c.k[page, :, t % PAGE] = nan
        c.v[page, :, t % PAGE] = nan
    c.call(lib)
    for s in range(len(ctx)):
        lo, hi = c.cu[s], c.cu[s + 1]
        assert torch.equal(c.out[lo:hi - 1], out[lo:hi - 1]) and torch.equal(c.lse[lo:hi - 1], lse[lo:hi - 1])
        assert bool(torch.isnan(c.out[hi - 1]).all()) and bool(torch.isnan(c.lse[hi - 1]).all())


def test_infinite_values_reach_only_rows_that_see_them(lib):
    c = Case([100, 190], [4, 3], seed=6).run(lib)
    out = c.out.clone()
    for s, t, d, x in [(0, 102, 5, float("inf")), (0, 103, 6, float("nan")), (1, 7, 9, float("inf")),
                       (1, 191, 8, float("-inf"))]:
        c.v[int(c.table[s, t // PAGE]), 1, t % PAGE, d] = x
    c.call(lib)
    want = torch.ones((7, H, D), dtype=torch.bool, device="cuda")
    heads = slice(16, 32)
    want[2:4, heads, 5] = False
    want[3:4, heads, 6] = False
    want[4:, heads, 9] = False
    want[5:, heads, 8] = False
    assert torch.equal(torch.isfinite(c.out), want)
    assert torch.equal(c.out[want], out[want])


def test_rows_of_minus_infinity_give_zeros(lib):
    c = Case([100, 3, 130], [2, 1, 3], seed=7)
    c.q.abs_().clamp_(min=0.01)
    for s in (0, 2):
        for p in range(pages(c.ctx[s] + c.nq[s])):
            c.k[int(c.table[s, p])] = float("-inf")
    t = 132  # ... but the last row of sequence 2 sees one finite score
    c.k[int(c.table[2, t // PAGE]), :, t % PAGE] = 0.5
    c.run(lib).check([1])
    assert bool((c.out[:2] == 0).all()) and bool((c.lse[:2] == float("-inf")).all())
    assert bool((c.out[3:5] == 0).all()) and bool((c.lse[3:5] == float("-inf")).all())
    v = c.v[int(c.table[2, t // PAGE]), :, t % PAGE].repeat_interleave(16, 0)
    assert torch.equal(c.out[5], v)


@pytest.mark.parametrize("kv", ["bf16", "fp8"])
@pytest.mark.parametrize("nq", [1, 2, 4, 8])
def test_maxima_that_keep_moving(lib, kv, nq):
    """Scores that grow along the cache: the running reference moves many times."""
    c = Case([1500], [nq], kv, seed=8, k_scale=1 / 64, v_scale=1 / 64, sm=0.5)
    n = 1500 + nq
    ramp = torch.linspace(0, 1, pages(n) * PAGE, device="cuda").view(-1, 1, PAGE, 1)
    qm = c.q.float().mean(0).view(G, 16, D).mean(1).view(1, G, 1, D)
    k = ramp * 4 * torch.sign(qm) + 0.05 * torch.randn((pages(n), G, PAGE, D), device="cuda")
    c.q.copy_((c.q.float() * 0.2 + torch.sign(qm).view(G, 1, D).expand(G, 16, D).reshape(1, H, D)).to(torch.bfloat16))
    ids = c.table[0].long()
    c.k[ids] = k.to(torch.bfloat16) if kv == "bf16" else (k * 64).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
    c.run(lib).check()


@pytest.mark.parametrize("kv", ["bf16", "fp8"])
@pytest.mark.parametrize("nq", [1, 2, 3, 8])
@pytest.mark.parametrize("at", [0, 5000, 9999])
@pytest.mark.parametrize("gap", [4.0, 9.0, 13.0])
def test_one_heavy_token_and_many_light_ones(lib, kv, nq, at, gap):
    """One token far above 10,000 equal ones, whose weights e^-gap are small but together count."""
    c = Case([10000], [nq], kv, seed=9, k_scale=1 / 64, v_scale=1 / 64, sm=1.0)
    c.q.zero_()
    c.q[:, :, 0] = 1.0
    ids = c.table[0].long()
    one = 1.0 if kv == "bf16" else 0x38  # a code of value 1 stands for 1/64
    c.k[ids] = 0
    c.k[int(c.table[0, at // PAGE]), :, at % PAGE, 0] = gap if kv == "bf16" else \
        int(torch.tensor(gap).to(torch.float8_e4m3fn).view(torch.uint8))
    if kv == "fp8":
        c.sm = 64.0
    c.v[ids] = one
    c.v[int(c.table[0, at // PAGE])] = 0
    c.run(lib).check()


@pytest.mark.parametrize("kv", ["bf16", "fp8"])
@pytest.mark.parametrize("sm", [0.0, -SM, 3.0])
def test_scales(lib, kv, sm):
    Case([700, 64], [1, 4], kv, seed=10, k_scale=1 / 64, v_scale=-1 / 64, sm=sm).run(lib).check()


@pytest.mark.parametrize("kv", ["bf16", "fp8"])
@pytest.mark.parametrize("nq", [1, 2, 4])
def test_queries_of_very_different_size(lib, kv, nq):
    """Heads of 1/256 and rows of 64 times the others' size, dims of 2^-20 and of zero."""
    c = Case([900], [nq], kv, seed=21, k_scale=1 / 64, v_scale=1 / 64)
    c.q[:, 5:64:9] *= 1 / 256
    c.q[nq - 1] *= 64
    c.q[:, :, 100:104] *= 2.0 ** -20
    c.q[:, :, 150:] = 0
    c.q[:, 33] = 0  # a head without a query: the mean of V
    c.run(lib).check()


@pytest.mark.parametrize("kv", ["bf16", "fp8"])
@pytest.mark.parametrize("bad", [float("inf"), float("-inf"), float("nan")])
def test_a_query_that_is_not_finite_stays_in_its_row_and_head(lib, kv, bad):
    c = Case([300], [4], kv, seed=22, k_scale=1 / 64, v_scale=1 / 64).run(lib)
    out, lse = c.out.clone(), c.lse.clone()
    c.q[2, 20, 7] = bad
    c.call(lib)
    keep = torch.ones((4, H), dtype=torch.bool, device="cuda")
    keep[2, 20] = False
    assert torch.equal(c.out[keep], out[keep]) and torch.equal(c.lse[keep], lse[keep])
    assert not bool(torch.isfinite(c.out[2, 20]).any()) and not bool(torch.isfinite(c.lse[2, 20]))


@pytest.mark.parametrize("kv", ["bf16", "fp8"])
@pytest.mark.parametrize("bad", [-1, -7, 1 << 20, 2147483647])
def test_bad_pages_take_no_part(lib, kv, bad):
    c = Case([1000, 300, 40], [1, 3, 1], kv, seed=11, k_scale=1 / 64, v_scale=1 / 64)
    good = c.table.clone()
    c.table[0, 7] = bad
    c.table[1, 4] = bad
    c.run(lib, code=lib.S5_ERR_DEVICE_BOUNDS)
    assert lib.s5_get_device_error(c.ws)[1] in (0, 1, 2, 3)
    c.table.copy_(good)  # (the expectation skips those pages)
    c.check([0, 2], {0: (7,)})
    # sequence 1's rows lose their own page; the earlier pages remain
    c.check([1], {1: (4,)})


@pytest.mark.parametrize("kv", ["bf16", "fp8"])
def test_bad_sequences_give_zeros(lib, kv):
    c = Case([100, 50, 60], [2, 1, 1], kv, seed=12, k_scale=1 / 64, v_scale=1 / 64)
    c.make(lib)
    for field, value in (("neg", -5), ("long", c.max_len)):
        c.batch.ctx_lens[1] = value
        c.out.fill_(7.0)
        c.call(lib)
        torch.cuda.synchronize()
        assert lib.s5_get_device_error(c.ws) == (lib.S5_ERR_DEVICE_BOUNDS, 2), field
        lib.s5_reset_device_error(c.ws)
        assert bool((c.out[2] == 0).all()) and bool((c.lse[2] == float("-inf")).all())
        c.check([0, 2])
    c.batch.ctx_lens[1] = 50
    # offsets that leave the rows: nothing outside [0, total_q) is written, sequence 0 is right
    c.batch.cu_q.copy_(torch.tensor([0, 2, 9, 4], dtype=torch.int32))
    c.call(lib)
    torch.cuda.synchronize()
    assert lib.s5_get_device_error(c.ws)[0] == lib.S5_ERR_DEVICE_BOUNDS
    c.check([0])


def test_pages_past_32_bit_offsets(lib):
    """Pools of more than 2^32 bytes and 2^31 values: the last pages are read."""
    n_pages = 44000
    c = Case([100], [1], seed=13)
    k, v = (torch.empty((n_pages, G, PAGE, D), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    high = torch.tensor([43999, 43800], dtype=torch.int32, device="cuda")
    ids = c.table[0].long()
    k[high.long()], v[high.long()] = c.k[ids], c.v[ids]
    c.k, c.v = k, v
    c.table.copy_(high[None])
    c.run(lib).check()


@pytest.mark.parametrize("kv", ["bf16", "fp8"])
def test_captured_and_replayed_with_other_lengths(lib, kv):
    c = Case([3000, 400, 64], [1, 2, 1], kv, seed=14, k_scale=1 / 64, v_scale=1 / 64).run(lib).check()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        c.call(lib)
        c.call(lib)
    for ctx in ([3000, 400, 64], [10, 0, 65], [2999, 430, 1]):
        c.ctx = ctx
        c.batch.ctx_lens.copy_(torch.tensor(ctx, dtype=torch.int32))
        c.q.copy_(torch.randn_like(c.q.float()).to(torch.bfloat16))
        c.out.fill_(9.0)
        graph.replay()
        torch.cuda.synchronize()
        c.check()
    assert lib.s5_get_device_error(c.ws)[0] == 0


def test_other_stream_and_shared_workspace(lib):
    """A call on another stream; batches of several shapes take turns in one workspace."""
    cs = [Case([9000, 40], [1, 1], seed=15).make(lib), Case([100] * 40, [4] * 40, "fp8", seed=16, k_scale=1 / 64,
                                                            v_scale=1 / 64).make(lib),
          Case([0, 300], [8, 20], seed=17).make(lib)]
    ws = max((c.ws for c in cs), key=lambda w: w.numel())
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    for c in cs + cs[::-1]:
        c.ws = ws
        c.call(lib, stream=st)
    st.synchronize()
    for c in cs:
        c.check()
    assert lib.s5_get_device_error(ws)[0] == 0


@pytest.mark.parametrize("kv", ["bf16", "fp8"])
@pytest.mark.parametrize("max_q", [1, 2, 3, 50])
def test_max_q_need_not_be_tight(lib, kv, max_q):
    """max_q chooses the rows of a tile; any value gives every row its answer."""
    c = Case([300, 64, 0, 900], [5, 1, 3, 2], kv, seed=19, k_scale=1 / 64, v_scale=1 / 64)
    c.max_q = max_q
    c.run(lib).check()


@pytest.mark.parametrize("kv", ["bf16", "fp8"])
@pytest.mark.parametrize("ctx,nq", [([5000, 64, 0], [1, 1, 1]), ([3000, 70], [4, 2])])
def test_expired_wait_is_reported_and_the_next_call_is_right(lib, kv, ctx, nq):
    """The test hook makes every CTA wait 1 ms for nothing: the call ends with S5_ERR_TIMEOUT."""
    c = Case(ctx, nq, kv, seed=20, k_scale=1 / 64, v_scale=1 / 64).run(lib).check()
    out = c.out.clone()
    at = lib.S5_WS_TEST_STALL_OFFSET
    c.ws[at:at + 8] = torch.tensor([1_000_000], dtype=torch.int64).view(torch.uint8).cuda()
    c.call(lib)
    torch.cuda.synchronize()
    assert lib.s5_get_device_error(c.ws)[0] == lib.S5_ERR_TIMEOUT
    lib.s5_reset_device_error(c.ws)
    c.out.fill_(9.0)
    c.call(lib)
    assert torch.equal(c.out, out)
    assert lib.s5_get_device_error(c.ws)[0] == 0


def test_equals_sparse_attention_over_every_block(lib):
    """With every history block selected, the sparse layer's answer is the dense one."""
    c = Case([2000, 700], [1, 1], seed=18).run(lib).check()
    topk = 512
    sel = torch.full((2, topk), -1, dtype=torch.int32, device="cuda")
    cnt = torch.tensor([2000 // 8, 700 // 8], dtype=torch.int32, device="cuda")
    for r in range(2):
        sel[r, :cnt[r]] = torch.arange(int(cnt[r]), device="cuda")
    out, lse = torch.empty_like(c.out), torch.empty_like(c.lse)
    lib.s5_sparse_gqa_attn(c.k, c.v, c.batch, c.q, sel, cnt, topk, SM, out, lse, c.ws)
    for s in range(2):
        _, _, tol, tol_lse = c.expect(s)
        assert bool(((out - c.out)[s].double().abs() <= 2 * tol[0]).all())
        assert bool(((lse - c.lse)[s].double().abs() <= 2 * tol_lse[0]).all())
