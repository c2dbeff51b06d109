"""kvx_shared_attention refuses strides that lead past any memory: their products are not to wrap round (no GPU
is needed)."""
import pytest

from tests.test_attention_abi import A, INV, attn_args, lib, pool  # noqa: F401


@pytest.mark.parametrize("which", ["q", "out"])
@pytest.mark.parametrize("kw", [dict(n_q=2 ** 27, q_heads=8, token=2 ** 40, head=64),
                                dict(n_q=8, q_heads=2 ** 27, token=64, head=2 ** 40)])
def test_strides_past_any_memory(lib, which, kw):  # noqa: F811
    p = pool()
    a = attn_args(n_q=kw["n_q"], q_heads=kw["q_heads"],
                  **{which + "_token_stride": kw["token"], which + "_head_stride": kw["head"]})
    assert lib.kvx_shared_attention(p.handle, a, A, 0, A, None) == INV
