"""Shared attention over 4-bit pools whose values are small beside the weights' range, or far apart in size.

The weights of keys behind a dominant one are small, and so are their products with small scales: a product has to
keep its 11 bits all the same.  The bounds are those of tests/attention_q4_ref.py, which counts two roundings a key, each of
at most 2^-11, and nothing absolute."""
import numpy as np
import pytest
import torch

from tests import attention_q4_ref as q4

pytestmark = pytest.mark.gpu


def _behind_sinks(D, step, gap):
    """Every 16th key has the score gap * ln 2 and a value of 0, all others the score 0 and values of 0 to 15 steps."""
    def edit(b):
        pair = b[..., D // 2:].view(np.float16)
        b[:, 0] = 0
        pair[:, 1, :, 0::2], pair[:, 1, :, 1::2] = step, 0
        b[::16, 1] = 0
        pair[::16, 0, :, 1::2] = gap * np.log(2) / np.sqrt(D)
    return edit


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("step", [2.0 ** -12, 2.0 ** -15 * 1.25, 2.0 ** -16 * 1.4375, 2.0 ** -17 * 1.4375, 2.0 ** -18 * 1.1875])
@pytest.mark.parametrize("gap", [8, 14, 17])
@pytest.mark.parametrize("qlens", [None, [3]])
def test_small_values_behind_dominant_keys(D, step, gap, qlens):
    c = q4.make("f16", "planes", 16, 2, G=2, D=D, lens=[4000], qlens=qlens, prefix=0, layers=1, layer=0,
                edit_bytes=_behind_sinks(D, step, gap))
    c.q[:] = 1
    c.v_scale = 2.0 ** 20  # (results in f16's normal range)
    q4.check(c, q4.Run(c).call().results())


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("by", [-6, -10, -13])
def test_small_values(D, by):
    """The usual values times a power of two (what subnormal scales become of it is what the pool then holds)."""
    def edit(b):
        pair = b[:, 1, :, D // 2:].view(np.float16)
        pair[:] = pair * np.float16(2.0 ** by)
    c = q4.make("f16", "planes", 16, 2, G=4, D=D, lens=[500, 61, 900], prefix=30, edit_bytes=edit)
    c.v_scale = 2.0 ** -by
    q4.check(c, q4.Run(c).call().results())


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("prefix", [0, 517])
@pytest.mark.parametrize("least,gap", [(-5, 14), (-9, 14), (-9, 20), (-12, 24)])
def test_a_great_scale_of_little_weight(D, prefix, least, gap):
    """One key's values have a scale of 4096 and next to no weight; the others are small and all alike in scale."""
    def edit(b):
        if len(b) < 40:
            return
        pair = b[..., D // 2:].view(np.float16)
        pair[:, 1, :, 0::2], pair[:, 1, :, 1::2] = 2.0 ** least * 0.1875, 0
        pair[33, 1, :, 0::2], pair[33, 1, :, 1::2] = 4096, -30000
        b[33, 0] = 0
        pair[33, 0, :, 1::2] = -gap * np.log(2) / np.sqrt(D)
    c = q4.make("f16", "planes", 16, 1, G=4, D=D, lens=[3000, 900], prefix=prefix, layers=1, layer=0, edit_bytes=edit)
    c.q[:] = 1
    c.v_scale = 2.0 ** (-least - 2)
    q4.check(c, q4.Run(c).call().results())
