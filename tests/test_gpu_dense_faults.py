"""Dense attention of batches whose offsets or lengths are wrong: zeros in the rows of the bad
sequences, the other sequences' rows as they would be without them."""
import pytest
import torch

from tests.test_gpu_dense import Case

pytestmark = pytest.mark.gpu


def run_with_wrong_offsets(lib, c, cu, zero_rows, good, left=(), ctx=None, times=20):
    """Calls with the offsets `cu` (and cached lengths `ctx`) again and again: the sequences `good` get
    their answers, `zero_rows` zeros, `left` stays as it was."""
    c.make(lib)
    c.batch.cu_q.copy_(torch.tensor(cu, dtype=torch.int32))
    if ctx is not None:
        c.batch.ctx_lens.copy_(torch.tensor(ctx, dtype=torch.int32))
    first = None
    for _ in range(times):
        c.out.fill_(7.0)
        c.lse.fill_(7.0)
        c.call(lib)
        torch.cuda.synchronize()
        assert lib.s5_get_device_error(c.ws)[0] == lib.S5_ERR_DEVICE_BOUNDS
        lib.s5_reset_device_error(c.ws)
        zero_rows, left = list(zero_rows), list(left)
        assert bool((c.out[zero_rows] == 0).all()) and bool((c.lse[zero_rows] == float("-inf")).all())
        assert bool((c.out[left] == 7.0).all()) and bool((c.lse[left] == 7.0).all())
        if first is None:
            first = c.out.clone(), c.lse.clone()
            c.check(good)
        assert torch.equal(c.out, first[0]) and torch.equal(c.lse, first[1])


# offsets of the batch, new tokens of its sequences, offsets given, rows of zeros, good sequences
WRONG = {
    "past_the_rows": ([2, 1, 1, 1], [0, 2, 9, 4, 5], [2, 3], [0, 3]),
    "negative": ([1, 1, 1, 1], [0, 1, -7, 3, 4], [1, 2], [0, 3]),
    "last": ([2, 3], [0, 2, 6], [2, 3, 4], [0]),
    "first": ([2, 3, 1], [-1, 2, 5, 6], [0, 1], [1, 2]),
    "two_of_them": ([1, 2, 1, 2, 1, 1], [0, 1, 2 ** 31 - 1, 4, -2 ** 31, 7, 8], [1, 2, 3, 4, 5, 6], [0, 5]),
}


@pytest.mark.parametrize("kv", ["bf16", "fp8"])
@pytest.mark.parametrize("long", [0, 2500])
@pytest.mark.parametrize("name", list(WRONG))
def test_wrong_offsets_leave_the_other_rows(lib, name, long, kv):
    nq, cu, zero_rows, good = WRONG[name]
    c = Case([long + 50 * (s % 3) for s in range(len(nq))], nq, kv, seed=40, k_scale=1 / 64, v_scale=1 / 64)
    run_with_wrong_offsets(lib, c, cu, zero_rows, good)


@pytest.mark.parametrize("n,at", [(40, (20,)), (700, (300,)), (3300, (5, 1600, 3299))])
@pytest.mark.parametrize("value", [-5, 1 << 30])
def test_wrong_offsets_in_large_batches(lib, n, at, value):
    """More sequences than a warp or one round of the prefix sums takes."""
    c = Case([s % 90 for s in range(n)], [1] * n, seed=41)
    cu = list(range(n + 1))
    for i in at:
        cu[i] = value
    zero_rows = sorted({r for i in at for r in (i - 1, i) if r < n})
    good = [s for s in range(n) if s not in zero_rows]
    run_with_wrong_offsets(lib, c, cu, zero_rows, good[:: max(1, n // 60)] + [r + d for r in zero_rows for d in (-1, 1)
                                                                              if r + d in good], times=10)


@pytest.mark.parametrize("kv", ["bf16", "fp8"])
def test_wrong_lengths_beside_wrong_offsets(lib, kv):
    """Sequence 2 (rows 2 to 4) has too many cached tokens, the offsets then fall back to 4, and sequence
    4 has rows 4 to 6: zeros in rows 2 and 3, sequence 4's answer in row 4 every time."""
    c = Case([100, 50, 60, 70, 80], [1, 1, 3, 2, 1], kv, seed=42, k_scale=1 / 64, v_scale=1 / 64)
    run_with_wrong_offsets(lib, c, [0, 1, 2, 5, 4, 7], [2, 3], [0, 1], left=[7], ctx=[100, 50, c.max_len, 70, 80])
    assert bool((c.lse[4:7] > float("-inf")).all())


@pytest.mark.parametrize("bad", [0, 31, 32, 1599, 3200])
def test_wrong_lengths_in_large_batches(lib, bad):
    n = 3201
    ctx = [s % 90 for s in range(n)]
    c = Case(ctx, [1] * n, seed=43)
    ctx = list(ctx)
    ctx[bad] = -1
    good = [s for s in range(0, n, 60) if s != bad] + [s for s in (bad - 1, bad + 1) if 0 <= s < n]
    run_with_wrong_offsets(lib, c, c.cu, [bad], good, ctx=ctx, times=10)
