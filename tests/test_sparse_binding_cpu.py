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
