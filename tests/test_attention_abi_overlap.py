"""kvx_shared_attention refuses results anywhere in the pool (no GPU is needed)."""
import pytest

from disaggregated_paged_kv_gb300 import kvx
from tests.test_attention_abi import A, attn_args, lib, pool  # noqa: F401

PLANE = 160 * 256


@pytest.mark.parametrize("layer", [0, 1])
@pytest.mark.parametrize("plane", [0, 1, 2, 3])
def test_results_in_any_plane(lib, layer, plane):  # noqa: F811
    p = pool()
    size = kvx.attention_workspace_size(p, 5, 3, 8, 32)
    for at in (plane * PLANE, (plane + 1) * PLANE - 2):
        a = attn_args(layer=layer, out=A + at)
        assert lib.kvx_shared_attention(p.handle, a, A, size, A, None) == kvx.ERR_OVERLAP
    # a first element before the pool, the last one in it
    a = attn_args(layer=layer, out=A - 2 * (4 * 512 + 7 * 64 + 63))
    assert lib.kvx_shared_attention(p.handle, a, A, size, A, None) == kvx.ERR_OVERLAP
