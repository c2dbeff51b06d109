"""kvx_shared_attention refuses prefixes of more positions than KVX_ATTN_MAX_POSITIONS (no GPU is needed)."""
import re
import os

from disaggregated_paged_kv_gb300 import kvx
from tests.test_attention_abi import A, INV, attn_args, lib, pool  # noqa: F401


def test_longest_prefix(lib):  # noqa: F811
    p, most = pool(), kvx.ATTN_MAX_POSITIONS
    assert kvx.attention_workspace_size(p, 5, 3, 8, most) > 0
    for bad in (most + 1, 2 ** 31 - 1):
        assert kvx.attention_workspace_size(p, 5, 3, 8, bad) == 0
        a = attn_args(prefix_len=bad, n_prefix_pages=2 ** 27)
        assert lib.kvx_shared_attention(p.handle, a, A, 1 << 40, A, None) == INV


def test_constant_is_the_headers():
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    with open(os.path.join(root, "include", "kvx.h")) as f:
        m = re.search(r"#define KVX_ATTN_MAX_POSITIONS (\d+)", f.read())
    assert int(m.group(1)) == kvx.ATTN_MAX_POSITIONS
