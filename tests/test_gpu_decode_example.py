"""The decode example end to end: transfer, block tables, scatter and shared attention together."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kw", [dict(), dict(requests=1, prefix_pages=0, steps=20),
                                dict(requests=40, prefix_pages=3, page=24, heads=4, group=7, dim=64, steps=30),
                                dict(requests=9, page=1, prefix_pages=33, dim=48, heads=3, group=1)])
def test_decode_example(kw):
    from examples import decode_step
    got, want = decode_step.run(**kw)
    for a, b in zip(got, want):
        # weights and results rounded to bf16 (2^-8 each) of values whose weighted mean size is below 1
        assert float((a.double() - b).abs().max()) < 2 * 2.0 ** -8 * float(b.abs().max() + 1)
