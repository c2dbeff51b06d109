"""kvx.shared_attention with scales so small that scores hardly differ, and queries that are 0 or nearly so."""
import pytest
import torch

from tests import attention_ref as ar

pytestmark = pytest.mark.gpu

ROOM = 300_000  # see test_gpu_attention.py


@pytest.mark.parametrize("dtype,io", [("fp8", torch.bfloat16), ("fp8", torch.float16), ("bf16", None), ("f16", None)])
@pytest.mark.parametrize("scale", [2.0 ** -3, 2.0 ** -24, 2.0 ** -40, 2.0 ** -120])
@pytest.mark.parametrize("room", [0, ROOM])
def test_zero_and_tiny_queries(dtype, io, scale, room):
    """Rows of zeros, of the smallest numbers of their type, and of ordinary ones, in narrow and wide tiles."""
    def edit(c):
        c.q[::3] = 0.0
        c.q[1::3, ::2] = torch.finfo(c.io).tiny
        c.q[5] = 0.0
        c.q[5, 0, 7] = torch.finfo(c.io).smallest_normal
    c = ar.make(dtype, "planes", 16, 1, 4, 64, lens=[230, 140, 29, 0, 300], qlens=[100, 90, 1, 1, 40], prefix=20,
                scale=scale, edit=edit, room=room, io=io)
    r = ar.Run(c)
    ar.check(c, r.call().results())
