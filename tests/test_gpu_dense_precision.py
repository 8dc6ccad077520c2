"""Dense attention held to the precision that its kernels state, and every page of V to its place.

The tolerances of tests/test_gpu_dense.py allow bf16 weights 2^-8 of A = sum_j w_j |V_j|; over a long cache
that hides the loss of a weight's second term and of whole pages.  Here:

- bf16 weights are two bf16 terms, each cut toward zero.  The first leaves 16 of a weight's 24 bits, of which
  the second keeps the upper 8 or more, so less than 2^8 steps of 2^-23 of the weight's power of two are
  lost: 2^-15 of the weight, and 2^-15 A in the sum.
- "balanced" values: V = +1 at the tokens whose weight loses most when only its upper 8 bits are kept and a
  constant below 0 at the others, chosen so that the row's sum nearly vanishes.  The rounding of the result is
  small there, and the loss of the second term is not.  Scores are one product q K with q = 1, in [-1, 0]; each
  page's first token has score 0, so that weights are relative to 1 whatever run of pages they are in.
- "marked" pages: q = 0, so every weight is a power of two, and V of page p is a whole number in dimension p % 192
  and 0 elsewhere.  Sums of whole numbers below 2^24 are exact; what remains is the quotient (2^-22) and
  the rounding of the result (2^-8).  A page left out or read twice is seen in its dimension.
"""
import math

import pytest
import torch

from tests.test_gpu_dense import BATCHES, D, G, PAGE, Case, pages

gpu = pytest.mark.gpu
TWO_TERMS, ONE_BYTE_2, ONE_BYTE_4 = 2.0 ** -15, 2.0 ** -11, 2.0 ** -9


# ---------------------------------------------------------------- any batch

@gpu
@pytest.mark.parametrize("name", list(BATCHES))
def test_bf16_weights_have_two_terms(lib, name):
    ctx, nq = BATCHES[name]
    c = Case(ctx, nq, seed=60 + len(name)).run(lib).check()
    v = c.v
    for s in range(len(ctx)):
        if nq[s] == 0:
            continue
        out, _, tol, _ = c.expect(s)
        c.v = v.abs()
        a = c.expect(s)[0]
        c.v = v
        lo, hi = c.cu[s], c.cu[s + 1]
        over = ((c.out[lo:hi].double() - out).abs() / (tol - (2.0 ** -8 - TWO_TERMS) * a)).max().item()
        assert over <= 1, (s, over)


# ---------------------------------------------------------------- balanced values

def balanced(n, one_byte, seed):
    """Scores x [n] and values v [n] (as the cache holds them), in 64 bits."""
    g = torch.Generator().manual_seed(seed)
    if one_byte:  # x = -code / 64, v = code / 64, E4M3 codes
        x = -(torch.rand(n, generator=g) * 64).to(torch.float8_e4m3fn).double() / 64
    else:
        x = -torch.rand(n, generator=g).to(torch.bfloat16).double()
    x[::PAGE] = 0
    w = torch.exp(x)
    loss = 1 - torch.exp(torch.frexp(w)[1].double() * math.log(2)) / 256 * torch.floor(
        torch.frexp(w)[0] * 256) / w
    high = loss > loss.median()
    v = torch.where(high, 1.0, -float((w * high).sum() / (w * ~high).sum()))
    v = (v * 64).float().to(torch.float8_e4m3fn).double() / 64 if one_byte else v.to(torch.bfloat16).double()
    # the rounding of the constant leaves a rest: whole values off until it is small
    idx = torch.nonzero(high)[:, 0]
    rest = (w * v).sum()
    for i in idx.tolist():
        if abs(rest) < 1:
            break
        if rest > 0:
            rest -= w[i] * v[i]
            v[i] = 0
        else:
            j = int(torch.nonzero(~high & (v != 0))[0])
            rest -= w[j] * v[j]
            v[j] = 0
    return x, v


def answer(x, v, n, weight):
    """out and its tolerance over the first n tokens."""
    w = torch.exp(x[:n])
    out, a = (w * v[:n]).sum() / w.sum(), (w * v[:n].abs()).sum() / w.sum()
    b = x[:n].abs().max()
    return float(out), float(2.0 ** -8 * out.abs() + (weight + 2 * (200 * 2.0 ** -24 * b + 2.0 ** -20) +
                                                      2.0 ** -27 * n + 2.0 ** -20) * a)


@pytest.mark.parametrize("n", [130, 700, 20000])
def test_one_term_is_not_enough(n):
    """The tolerance tells two terms from one (the formula with weights cut to their terms; no GPU)."""
    x, v = balanced(n, False, n)
    w = torch.exp(x).float()
    first = (w.view(torch.int32) & -65536).view(torch.float32)
    second = ((w - first).view(torch.int32) & -65536).view(torch.float32)
    out, tol = answer(x, v, n, TWO_TERMS)
    total = w.double().sum()
    assert abs(float((first.double() * v).sum() / total) - out) > 2 * tol
    assert abs(float(((first.double() + second.double()) * v).sum() / total) - out) <= tol


@gpu
@pytest.mark.parametrize("kv", ["bf16", "fp8"])
@pytest.mark.parametrize("nq", [1, 2, 4, 6])
@pytest.mark.parametrize("n", [130, 700, 20000])
def test_balanced_values(lib, n, nq, kv):
    """Row r of nq sees n - nq + r + 1 tokens."""
    one = kv == "fp8"
    x, v = balanced(n, one, n)
    c = Case([n - nq], [nq], kv, seed=61, k_scale=1 / 64, v_scale=1 / 64, sm=1.0)
    ids = c.table[0].long()

    def put(pool, y, dims):
        z = torch.zeros((pages(n) * PAGE, D), dtype=torch.float32)
        z[:n, dims] = y.float()[:, None] * (64 if one else 1)
        z = z.to(torch.float8_e4m3fn).view(torch.uint8) if one else z.to(torch.bfloat16)
        pool[ids] = z.view(-1, 1, PAGE, D).expand(-1, G, -1, -1).cuda()

    put(c.k, x, slice(0, 1))
    put(c.v, v, slice(0, D))
    c.q.zero_()
    c.q[:, :, 0] = 1.0
    c.run(lib)
    weight = TWO_TERMS if not one else ONE_BYTE_2 if nq <= 2 else ONE_BYTE_4
    for r in range(nq):
        out, tol = answer(x, v, n - nq + r + 1, weight)
        assert float((c.out[r].double() - out).abs().max()) <= tol, r


# ---------------------------------------------------------------- marked pages

@gpu
@pytest.mark.parametrize("kv", ["bf16", "fp8"])
@pytest.mark.parametrize("ctx,nq", [([70000], [1]), ([70000], [2]), ([70000], [4]), ([33000, 20000], [7, 1]),
                                    ([(977 * i) % 6000 for i in range(70)], [1 + i % 4 for i in range(70)]),
                                    ([(37 * i) % 400 for i in range(200)], [1] * 200)])
def test_every_page_in_its_place(lib, ctx, nq, kv):
    one = kv == "fp8"
    c = Case(ctx, nq, kv, seed=62, k_scale=1 / 64, v_scale=2.0 if one else 1.0)
    value = torch.zeros((c.v.shape[0], G, D), device="cuda")  # of all tokens of a page
    for s in range(len(ctx)):
        p = torch.arange(pages(ctx[s] + nq[s]), device="cuda")
        for g in range(G):
            value[c.table[s, p].long(), g, (p + 48 * g) % D] = ((p // D + p + g + s) % 7 + 1).float()
    v = value[:, :, None].expand(-1, -1, PAGE, -1)
    c.v = (v.to(torch.float8_e4m3fn).view(torch.uint8) if one else v.to(torch.bfloat16)).contiguous()
    c.q.zero_()
    c.run(lib)
    for s in range(len(ctx)):
        of_page = value[c.table[s, :pages(ctx[s] + nq[s])].long()].double()  # [pages][G][D]
        for r in range(nq[s]):
            n = ctx[s] + r + 1
            seen = (n - PAGE * torch.arange(of_page.shape[0], device="cuda")).clamp(0, PAGE).double()
            want = ((of_page * seen[:, None, None]).sum(0) * c.v_scale / n).repeat_interleave(16, 0)
            got = c.out[c.cu[s] + r].double()
            assert bool(((got - want).abs() <= (2.0 ** -8 + 2.0 ** -20) * want).all()), (s, r)
            # (reference 0 or -12) + log2 of the sum, to 2^-22 of itself, the sum and the product rounded
            assert bool(((c.lse[c.cu[s] + r].double() - math.log(n)).abs() <= 2.0 ** -21 * (12 + math.log2(n))).all())
