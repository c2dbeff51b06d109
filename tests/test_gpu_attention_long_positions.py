"""kvx.shared_attention refuses lengths whose tiles would end past 32-bit positions, where the table has room
for them."""
import pytest
import torch

from disaggregated_paged_kv_gb300 import kvx
from tests import attention_ref as ar

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype,D", [("bf16", 64), ("fp8", 128), ("f32", 64)])
@pytest.mark.parametrize("n", [3, 80])
def test_lengths_near_2_to_the_31(dtype, D, n):
    """Table rows of 2^31 positions (pages of 20,000 tokens), with and without query starts."""
    c = ar.make(dtype, "planes", 20_000, 1, 4, D, lens=[40 + i % 9 for i in range(n)], prefix=20, layers=1,
                layer=0, room=2 ** 31)
    r = ar.Run(c)
    good = r.lens.clone()
    for q_start in (None, r.q_start):
        for length in (2 ** 31 - 1, 2 ** 31 - 63, kvx.ATTN_MAX_POSITIONS + 1):
            r.lens[n // 2] = length
            r.call(q_start=q_start)
            torch.cuda.synchronize()
            assert int(r.status.item()) == kvx.ERR_OUT_OF_RANGE
            r.lens.copy_(good)
            ar.check(c, r.call(q_start=q_start).results())
