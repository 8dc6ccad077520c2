"""``Batch`` refuses arrays that do not belong together: the kernels read, and the table call writes, a row of
the page table per sequence (no GPU needed: tensors that pass for CUDA tensors)."""
import pytest
import torch


class Cuda(torch.Tensor):
    is_cuda = True
    place = torch.device("cuda", 0)

    @property
    def device(self):
        return self.place


class Other(Cuda):
    place = torch.device("cuda", 1)


@pytest.fixture(scope="module")
def s5():
    from block_sparse_gqa_indexer_b200 import build
    build.build()
    from block_sparse_gqa_indexer_b200 import s5 as mod
    return mod


def _arrays(rows, n, kinds=(Cuda, Cuda, Cuda)):
    shapes = ((rows, 4), (n,), (n + 1,))
    return [torch.zeros(s, dtype=torch.int32).as_subclass(k) for s, k in zip(shapes, kinds)]


@pytest.mark.parametrize("rows,n", [(1, 2), (0, 1), (7, 8)])
def test_a_page_table_of_fewer_rows(s5, rows, n):
    with pytest.raises(ValueError, match=f"page_table has {rows} rows for {n} sequences"):
        s5.Batch(*_arrays(rows, n), 4, 1, 100)


@pytest.mark.parametrize("rows,n", [(2, 2), (9, 2)])
def test_tables_of_as_many_rows_or_more(s5, rows, n):
    b = s5.Batch(*_arrays(rows, n), 4, 1, 100)
    assert (b.desc.batch, b.desc.max_pages) == (n, 4)


@pytest.mark.parametrize("kinds", [(Cuda, Other, Cuda), (Cuda, Cuda, Other), (Other, Cuda, Cuda)])
def test_arrays_of_different_devices(s5, kinds):
    with pytest.raises(ValueError, match="cuda:1"):
        s5.Batch(*_arrays(2, 2, kinds), 4, 1, 100)
