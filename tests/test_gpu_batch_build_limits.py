"""``s5_build_batch`` at the largest sizes that its arguments allow."""
import pytest
import torch

pytestmark = pytest.mark.gpu


def test_rows_next_to_the_largest_32_bit_number(lib):
    """2^31 - 1 rows: 1,024 requests of 2^21 new tokens each, the last row cut off; nothing is written
    in front of the outputs or behind them."""
    n, length, pages, rows, pad = 1024, lib.MAX_LEN, lib.MAX_LEN // lib.PAGE, 2 ** 31 - 1, 1 << 18
    i32 = dict(dtype=torch.int32, device="cuda")
    req_pages, table = torch.full((n, pages), -1, **i32), torch.empty((n, pages), **i32)
    free = torch.arange(n * pages - 1, -1, -1, **i32)  # row r's page: n * pages - 1 - r / 64
    req_ids, ctx = torch.arange(n, **i32), torch.zeros(n, **i32)
    new, cu, used = torch.full((n,), length, **i32), torch.empty(n + 1, **i32), torch.empty(1, **i32)
    guarded = [torch.full((rows + 2 * pad,), -9, **i32) for _ in range(2)]
    slots, positions = (g[pad:pad + rows] for g in guarded)
    batch = lib.Batch(table, ctx, cu, rows, length, length)
    ws = torch.zeros(lib.S5_WS_FIXED_BYTES, dtype=torch.uint8, device="cuda")
    lib.s5_build_batch(req_pages, req_ids, new, free, batch, slots, positions, used, ws)
    assert lib.s5_get_device_error(ws) == (lib.S5_ERR_DEVICE_BOUNDS, n - 1)
    for g in guarded:
        assert bool((g[:pad] == -9).all()) and bool((g[-pad:] == -9).all())
    assert torch.equal(table.flatten(), free) and torch.equal(req_pages, table)
    assert used.item() == n * pages and cu.tolist() == [length * s for s in range(n)] + [rows]
    step = 1 << 26
    for first in range(0, rows, step):
        r = torch.arange(first, min(rows, first + step), device="cuda")
        page = n * pages - 1 - r // lib.PAGE
        slot = torch.where(page <= 2 ** 25 - 2, page * lib.PAGE + r % lib.PAGE, -1)
        assert torch.equal(slots[first:first + step], slot.to(torch.int32))
        assert torch.equal(positions[first:first + step], (r % length).to(torch.int32))
