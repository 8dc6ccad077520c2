"""Dense attention of batches with many sequences without new tokens between those with some (a batch whose
places are fixed, most of them empty): the right rows, and not the time of a dependent load per empty place."""
import pytest
import torch

from tests.test_gpu_dense import Case

pytestmark = pytest.mark.gpu


def with_holes(live, holes):
    """`live` (ctx, new) pairs with holes[i] empty sequences before pair i, and holes[-1] behind them."""
    ctx, nq = [], []
    for (c, n), h in zip(live + [(0, 0)], holes):
        ctx += [64 * (i % 2) for i in range(h)] + [c]
        nq += [0] * h + [n]
    return ctx[:-1], nq[:-1]


@pytest.mark.parametrize("kv", ["bf16", "fp8"])
@pytest.mark.parametrize("holes", [(0, 30, 31, 0), (5, 31, 32, 1), (33, 63, 64, 31), (0, 500, 1, 900), (2000, 0, 4000, 0)])
@pytest.mark.parametrize("nq", [1, 3])
def test_holes_of_any_length(lib, holes, nq, kv):
    """Gaps around multiples of 32, in batches that a warp, one round and several rounds of the sums take."""
    for long in (0, 2000):
        ctx, new = with_holes([(long + 70, nq), (3, 1), (long, nq)], holes)
        Case(ctx, new, kv, seed=50 + nq, k_scale=1 / 64, v_scale=1 / 64).run(lib).check(
            [s for s, n in enumerate(new) if n])


def test_holes_cost_little(lib):
    """3,000 empty places between two sequences: one read of L2 after the other, they cost more than 1 ms.
    (The first sequence has 4 * (141 + 2) units, both 768: a thread block's share of 6 lies over the places.)"""
    def best_us(holes):
        ctx, new = with_holes([(9000, 1), (3000, 1)], (0, holes, 0))
        c = Case(ctx, new, seed=51).run(lib)
        for _ in range(3):
            c.call(lib)
        best = float("inf")
        for _ in range(10):
            ev = [torch.cuda.Event(enable_timing=True) for _ in range(2)]
            ev[0].record()
            for _ in range(5):
                c.call(lib)
            ev[1].record()
            torch.cuda.synchronize()
            best = min(best, ev[0].elapsed_time(ev[1]) * 200)
        return best

    without, with_3000 = best_us(0), best_us(3000)
    assert with_3000 < without + 300, (without, with_3000)
