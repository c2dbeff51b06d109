"""What slots hold that no row sees does not reach a result, to the bit: shared attention over 4-bit pools whose
unseen slots hold zeros in one run and finite numbers at the ends of f16 in the others."""
import pytest
import torch

from tests import attention_q4_ref as q4
from tests import attention_q4_unseen as un

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kind,page", [("planes", 16), ("planes", 1), ("slots", 1), ("slots", 24), ("hnd", 16), ("hnd", 3)])
@pytest.mark.parametrize("D,H", [(64, 1), (64, 2), (128, 1), (128, 8)])
@pytest.mark.parametrize("qlens", [None, (3, 9, 1, 2)])
def test_slots_of_no_token(kind, page, D, H, qlens):
    """A prefix that ends within a block of keys, so that a request's first block begins below its own tokens;
    requests that end within a block.  Values of about 1e-3, which lose bits next to a great scale."""
    c = q4.make("f16", kind, page, H, G=4, D=D, lens=[211, 97, 130, 1100], qlens=qlens, prefix=77, seed=D,
                edit_bytes=un.small_values(D))
    v, unseen = un.no_token(c)
    assert int(unseen.sum()) > 0
    v[unseen] = un.vector(D, 0, 0, 0)
    want = un.run(c)
    q4.check(c, want)
    for ends in un.ENDS:
        v[unseen] = un.vector(D, *ends)
        for a, b in zip(want, un.run(c)):
            assert torch.equal(a, b)


@pytest.mark.parametrize("D", [64, 96, 128])
@pytest.mark.parametrize("page", [16, 1])
def test_a_prefix_longer_than_its_requests(D, page):
    """Positions of the prefix that no request reaches."""
    lens = [300 - 7 * (i % 6) for i in range(40)]
    c = q4.make("bf16", "planes", page, 2, G=4, D=D, lens=lens, prefix=517, seed=3, room=600, layers=1, layer=0,
                edit_bytes=un.small_values(D))
    pool, slots = c.pool.view(2, c.slots, 2, -1), un.slots(c, range(300, 517))
    pool[:, slots] = un.vector(D, 0, 0, 0)
    want = un.run(c)
    q4.check(c, want)
    for ends in un.ENDS:
        pool[:, slots] = un.vector(D, *ends)
        for a, b in zip(want, un.run(c)):
            assert torch.equal(a, b)
