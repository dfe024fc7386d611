"""How the binding describes tensors to the sparse decode calls, without a GPU: nothing is launched."""
import pytest

torch = pytest.importorskip("torch")


class OnGpu(torch.Tensor):
    """A host tensor that says it is a CUDA one."""
    is_cuda = True


def on_gpu(t):
    return t.as_subclass(OnGpu)


@pytest.fixture(scope="module")
def kvo():
    from gather_radix_top_gb300 import build, kvo as K
    build.build()
    return K


def rows(n=16):
    return on_gpu(torch.zeros(n, 656, dtype=torch.uint8))


@pytest.mark.parametrize("table", [torch.empty(2, 0, dtype=torch.int32), torch.zeros(2, 9, dtype=torch.int32)[:, 5:5],
                                   torch.empty(1, 0, dtype=torch.int32)])
def test_a_table_without_columns_is_a_table(kvo, table):
    """Torch gives an empty tensor the address 0, which would say that there is no table: sequence s were block s."""
    c = kvo.Cache(rows=rows(), block_rows=4, table=on_gpu(table)).c
    assert c.table and c.table % 4 == 0
    assert c.table_blocks == 0 and c.table_ld >= 0 and c.sequences == table.shape[0]
    full = kvo.Cache(rows=rows(), block_rows=4, table=on_gpu(torch.zeros(2, 9, dtype=torch.int32)[:, 5:6])).c
    assert full.table_blocks == 1 and full.table_ld == 9
    assert not kvo.Cache(rows=rows(), block_rows=4).c.table


def test_a_cache_of_no_sequences_is_refused(kvo):
    """A table without rows: the calls say what is wrong, before anything is launched."""
    table = on_gpu(torch.empty(0, 4, dtype=torch.int32))
    cache = kvo.Cache(rows=rows(), keys=on_gpu(torch.zeros(16, 128, dtype=torch.bfloat16)), block_rows=4, table=table)
    lens = on_gpu(torch.zeros(2, dtype=torch.int32))
    with pytest.raises(ValueError, match="sequences"):
        kvo.kvo_attend(0, cache, on_gpu(torch.zeros(2, 1, 576, dtype=torch.bfloat16)), lens, 0.1, rows=4)
    with pytest.raises(ValueError, match="sequences"):
        kvo.kvo_index_scores(0, cache, on_gpu(torch.zeros(2, 1, 128, dtype=torch.bfloat16)), on_gpu(torch.zeros(2, 1)), lens, 4)
