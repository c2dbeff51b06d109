"""Tables of a single row may come with any stride between rows, there being no second one."""
import pytest
import torch

from tests import attention_ref as ar
from tests import test_gpu_tables as tt

pytestmark = pytest.mark.gpu


def rows_of(x, stride):
    return torch.as_strided(x.contiguous().view(-1), x.shape, (stride, 1))


@pytest.mark.parametrize("stride", [0, 1, 3])
def test_attention(stride):
    c = ar.make("bf16", "planes", 16, 2, 4, 64, lens=[200], prefix=32)
    r = ar.Run(c)
    r.tables = rows_of(r.tables, stride)
    ar.check(c, r.call().results())


@pytest.mark.parametrize("stride", [0, 1, 3])
def test_block_tables(stride):
    c = tt.Call(16, [20], [200])
    c.d_tables = rows_of(c.d_tables, stride)
    c.check()


def test_transposed_column():
    c = tt.Call(16, [20], [200])
    column = c.d_tables.t().contiguous()
    c.d_tables = column.t()
    c.check()
