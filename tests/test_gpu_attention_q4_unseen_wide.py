"""Shared attention over 4-bit pools where many rows meet the same keys: values are made into 16-bit numbers there, and
what that makes of slots that a row does not see does not reach its result."""
import pytest
import torch

from tests import attention_q4_ref as q4
from tests import attention_q4_unseen as un

pytestmark = pytest.mark.gpu

# (with query starts the tables' room stands for the keys: small cases take the kernel of many rows)
ROOM = 600_000


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("page", [16, 1])
@pytest.mark.parametrize("reach", [300, 256, 383])
def test_a_prefix_longer_than_its_requests(D, page, reach):
    """Positions of the prefix that no row sees, though a request without query tokens reaches them."""
    lens = [reach - 7 * (i % 6) for i in range(40)]
    c = q4.make("bf16", "planes", page, 2, G=4, D=D, lens=lens + [530], qlens=[1] * 40 + [0], prefix=517, seed=3, room=ROOM,
                layers=1, layer=0)
    pool, slots = c.pool.view(2, c.slots, 2, -1), un.slots(c, range(reach, 517))
    pool[:, slots] = un.vector(D, 0, 0, 0)
    want = un.run(c)
    q4.check(c, want)
    for ends in un.ENDS:
        pool[:, slots] = un.vector(D, *ends)
        for a, b in zip(want, un.run(c)):
            assert torch.equal(a, b)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("ends", [(0, 0, 0), (0x6C00, 0, 0xFF), (0x7000, 0, 0xFF), (0x7000, 0xF380, 0xF0), (0x7BFF, 0x7BFF, 0xFF)])
@pytest.mark.parametrize("plane", [0, 1])
def test_tokens_that_only_later_rows_see(D, ends, plane):
    """The last three tokens of a prompt hold elements up to f16's end, and beyond it; a row that sees a value beyond has
    an infinity there and its other columns as ever."""
    c = q4.make("bf16", "planes", 16, 1, G=2, D=D, lens=[270], qlens=[200], prefix=0, layers=1, layer=0, room=ROOM)
    pool, slots = c.pool.view(2, c.slots, -1), un.slots(c, (266, 267, 269))
    want = un.run(c)
    q4.check(c, want)
    pool[plane, slots] = un.vector(D, *ends)
    got = un.run(c)
    for a, b in zip(want, got):
        assert torch.equal(a[:196], b[:196])
    if plane == 1:
        code = torch.tensor([ends[2] & 15, ends[2] >> 4] * (D // 2), dtype=torch.float64)
        num = lambda x: float(torch.tensor([x], dtype=torch.int32).to(torch.int16).view(torch.float16))  # noqa: E731
        v = code * num(ends[0]) + num(ends[1])
        beyond = v.abs() > 65520
        for j in (266, 267, 269):
            c.kv[0][j, 1, 0], c.mag[0][j, 1, 0] = v, code * abs(num(ends[0])) + abs(num(ends[1]))
        ref, _, tol, _ = q4.reference(c)
        q4.ar._near(got[0][196:][..., ~beyond], ref[196:][..., ~beyond], tol[196:][..., ~beyond], "out")
        assert bool((got[0][196:][..., beyond] == torch.inf * torch.sign(v[beyond])).all())
