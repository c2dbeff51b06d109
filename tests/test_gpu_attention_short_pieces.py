"""kvx.shared_attention where a CTA of the 128-row kernel has many pieces of one or two key tiles, so that
its loads run pieces ahead of its softmax: infinities and NaN in V that some rows of a tile see and others
do not reach exactly the rows that see them, and the same call gives the same bits."""
import math

import pytest
import torch

from tests import attention_ref as ar

pytestmark = pytest.mark.gpu

ROOM = 300_000  # see test_gpu_attention.py


def check_again_and_again(c, times=12):
    r = ar.Run(c)
    first = r.call().results()
    ar.check(c, first)
    bits = r.out.clone().view(torch.int16)
    for _ in range(times):
        r.out.fill_(1.0)
        r.call()
        r.results()
        assert torch.equal(r.out.view(torch.int16), bits)


@pytest.mark.parametrize("dtype,value", [("bf16", math.nan), ("bf16", math.inf), ("f16", -math.inf),
                                         ("f16", math.nan), ("fp8", math.nan)])
@pytest.mark.parametrize("n_lo,n_hi", [(60, 120), (100, 250)])
def test_short_prompts(dtype, value, n_lo, n_hi):
    """64 prompts of a tile of keys (or two), every second one with such a value in some token's V."""
    lens = [n_lo + (23 * i) % (n_hi - n_lo + 1) for i in range(64)]

    def edit(c):
        for b in range(0, len(lens), 2):
            c.kv[b][lens[b] - 1 - (7 * b) % 40, 1] = torch.tensor(value).to(c.kv[b].dtype)
    check_again_and_again(ar.make(dtype, "planes", 16, 8, 4, 64, lens=lens, qlens=[min(n, 90) for n in lens], prefix=0,
                                  layers=1, layer=0, edit=edit, room=ROOM))


@pytest.mark.parametrize("dtype", ["bf16", "fp8"])
@pytest.mark.parametrize("prefix", [120, 250])
def test_short_prefix_of_many_rows(dtype, prefix):
    """870 single tokens behind a prefix whose late positions hold NaN values: requests shorter than that do
    not see them."""
    lens = [20 + (37 * i) % (prefix + 30) for i in range(870)]

    def edit(c):
        for x in [c.common] + c.kv:
            x[prefix - 21:, 1] = torch.tensor(math.nan).to(x.dtype)
    check_again_and_again(ar.make(dtype, "planes", 16, 16, 8, 64, lens=lens, prefix=prefix, layers=1, layer=0,
                                  edit=edit, room=ROOM, starts=True), 6)
