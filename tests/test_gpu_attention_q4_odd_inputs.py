"""Shared attention over 4-bit pools with infinities and NaN in places that are seen: they stay where they belong."""
import math

import pytest
import torch

from tests import attention_q4_ref as q4
from tests import attention_q4_unseen as un

pytestmark = pytest.mark.gpu

ROOM = 600_000


@pytest.mark.parametrize("D", [64, 96, 128])
@pytest.mark.parametrize("what", [0x7C00, 0xFC00, 0x7E00])
@pytest.mark.parametrize("at,qlens", [(37, None), (79, None), (37, [3]), (5, [70])])
def test_a_seen_scale_that_is_not_finite(D, what, at, qlens):
    """One group of one key's values: its columns are not finite, all others are as ever."""
    c = q4.make("bf16", "planes", 16, 1, G=4, D=D, lens=[80], qlens=qlens, prefix=0, layers=1, layer=0, room=ROOM if qlens else 0)
    pool, (slot,) = c.pool.view(2, c.slots, D // 8 * 5), un.slots(c, [at])
    pool[1, slot, D // 2 + 4:D // 2 + 6] = torch.tensor([what & 255, what >> 8], dtype=torch.uint8)  # scale of group 1
    out, lse = q4.Run(c).call().results()
    want, wlse, tol, tol_l = q4.reference(c)
    keep = [i for i in range(D) if not 32 <= i < 64]
    q4.ar._near(out[..., keep], want[..., keep], tol[..., keep], "out")
    q4.ar._near(lse, wlse, tol_l, "lse")
    sees = torch.tensor([80 - c.T + t + 1 > at for t in range(c.T)])
    assert not bool(torch.isfinite(out[sees][..., 32:64]).any())
    q4.ar._near(out[~sees], want[~sees], tol[~sees], "rows that do not see it")


@pytest.mark.parametrize("D", [64, 96, 128])
@pytest.mark.parametrize("what", [math.nan, math.inf, -math.inf, 3e38])
@pytest.mark.parametrize("lens,qlens,prefix,room", [([300, 161, 200], None, 150, 0), ([300], [5], 0, 0), ([300, 310], [90, 100], 40, ROOM)])
def test_a_query_row_that_is_not_finite(D, what, lens, qlens, prefix, room):
    c = q4.make("bf16", "planes", 16, 2, G=2, D=D, lens=lens, qlens=qlens, prefix=prefix, room=room)
    want = un.run(c)
    q4.check(c, want)
    c.q[1, 1, 3] = what
    for a, b in zip(want, un.run(c)):
        a[1, 1], b[1, 1] = 0, 0
        assert torch.equal(a, b)
