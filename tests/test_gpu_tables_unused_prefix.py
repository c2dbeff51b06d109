"""kvx.block_tables looks at the shared prefix's page ids only where a new request uses them."""
import pytest

from disaggregated_paged_kv_gb300 import kvx
from tests.test_gpu_tables import Call

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("n", [2, 1024, 1500])
@pytest.mark.parametrize("bad", [-1, 10 ** 6])
def test_prefix_ids_without_a_new_request(n, bad):
    """Running requests and padding rows: garbage in the prefix list is not used."""
    c = Call(16, [33, 64, 0, 70][:n] + [40] * (n - 4), [34, 70, 0, 71][:n] + [41] * (n - 4), prefix=2)
    c.d_prefix[1] = bad
    c.check()


@pytest.mark.parametrize("n", [4, 1500])
def test_prefix_ids_with_one(n):
    for b in (0, n - 1):
        old, new = [40] * n, [41] * n
        old[b], new[b] = 0, 50
        c = Call(16, old, new, prefix=2)
        before = [x.clone() for x in (c.d_tables, c.d_q, c.d_slots)]
        c.d_prefix[1] = -1
        assert c.run() == kvx.ERR_OUT_OF_RANGE
        for x, y in zip(before, (c.d_tables, c.d_q, c.d_slots)):
            assert x.equal(y)
