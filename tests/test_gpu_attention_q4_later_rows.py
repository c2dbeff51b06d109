"""Drafts over a 4-bit pool: a row's result does not depend, to the bit, on the tokens behind it."""
import pytest
import torch

from tests import attention_q4_ref as q4
from tests import attention_q4_unseen as un

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("G,lens,qlens,prefix", [(2, [70], [6], 0), (1, [1500], [8], 0), (4, [39], [2], 0), (8, [200], [30], 0),
                                                 (3, [131], [5], 70), (1, [19], [8], 0)])
@pytest.mark.parametrize("plane", [0, 1])
def test_tokens_that_only_later_rows_see(D, G, lens, qlens, prefix, plane):
    """The last two tokens' keys or values are as great as they can be."""
    c = q4.make("bf16", "planes", 16, 1, G=G, D=D, lens=lens, qlens=qlens, prefix=prefix, layers=1, layer=0,
                edit_bytes=un.small_values(D))
    pool = c.pool.view(2, c.slots, -1)
    slots, before = un.slots(c, range(lens[0] - 2, lens[0])), qlens[0] - 2
    want = un.run(c)
    q4.check(c, want)
    for ends in [(0, 0, 0), (0x6C00, 0x0000, 0xFF), (0x6C00, 0xF380, 0xF0), (0x7BFF, 0x7BFF, 0xFF)]:
        pool[plane, slots] = un.vector(D, *ends)
        for a, b in zip(want, un.run(c)):
            assert torch.equal(a[:before], b[:before])


@pytest.mark.parametrize("D", [64, 128])
def test_requests_shorter_than_the_prefix(D):
    """Rows of one unit that see different stretches of a prefix: values behind a request's end are great."""
    lens = [40, 300, 77, 300, 300, 150]
    c = q4.make("bf16", "planes", 16, 1, G=1, D=D, lens=lens, prefix=290, layers=1, layer=0, edit_bytes=un.small_values(D))
    pool, slots = c.pool.view(2, c.slots, -1), un.slots(c, range(150, 290))
    want = un.run(c)
    q4.check(c, want)
    for plane in (0, 1):
        pool[plane, slots] = un.vector(D, 0x6C00, 0xF380, 0xF3)
        for a, b in zip(want, un.run(c)):
            for row in (0, 2, 5):
                assert torch.equal(a[row], b[row])
