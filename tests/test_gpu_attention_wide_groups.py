"""kvx.shared_attention with more query heads a kv head than the narrow kernel has rows (64): single tokens,
with and without query starts, few requests and so many that the call is planned without them."""
import pytest

from tests import attention_ref as ar

pytestmark = pytest.mark.gpu


def run(c, **more):
    r = ar.Run(c)
    ar.check(c, r.call(**more).results())


@pytest.mark.parametrize("dtype", ["bf16", "fp8"])
@pytest.mark.parametrize("n", [1, 40, 2100])
@pytest.mark.parametrize("starts", [False, True])
def test_single_tokens(dtype, n, starts):
    """2100 requests of 71 heads behind 128 shared tokens are 4.9e9 operations: the wide kernel's."""
    lens = [128 + 1 + (5 * i) % 30 for i in range(n)]
    if n > 1:
        lens[1] = 0
        lens[n // 2] = 77
    run(ar.make(dtype, "planes", 16, 1, 71, 64, lens=lens, prefix=128, layers=1, layer=0, starts=starts,
                room=20_000 if n == 40 else 0))


@pytest.mark.parametrize("G", [65, 100, 300])
def test_single_tokens_among_prompts(G):
    run(ar.make("bf16", "planes", 16, 1, G, 64, lens=[700, 301, 0, 640, 333, 650], qlens=[1, 30, 1, 1, 33, 5],
                prefix=300, room=100_000))


def test_query_starts_change_nothing():
    """Single tokens of 71 heads share the pass over the prefix whether or not their starts are given: the
    same tiles, and so the same bits."""
    lens = [128 + 1 + (5 * i) % 30 for i in range(2000)]
    c = ar.make("bf16", "planes", 16, 1, 71, 64, lens=lens, prefix=128, layers=1, layer=0)
    r = ar.Run(c)
    out, lse = r.call(q_start=None).results()
    with_starts = r.call(q_start=r.q_start).results()
    assert out.equal(with_starts[0]) and lse.equal(with_starts[1])
