"""The chain of kernels behind kvx.shared_attention with many rows over the prefix (plan, 128-row tiles, the
requests' own keys beside them, join): captured, on several streams, and call behind call with inputs that
the kernel just before has written."""
import pytest
import torch

from tests import attention_ref as ar

pytestmark = pytest.mark.gpu

ROOM = 300_000  # see test_gpu_attention.py: with query starts, the tables' room brings the wide kernel in


def planned(dtype, seed, turn=0):
    """Decode with query starts: 60 requests of 4 rows a kv head behind 512 shared tokens."""
    lens = [512 + 1 + 37 * (i % 7) for i in range(60)]
    lens[9] = 0
    return ar.make(dtype, "planes", 16, 2, 4, 128, lens=lens[turn:] + lens[:turn], prefix=512, layers=1, layer=0,
                   seed=seed, room=ROOM, starts=True)


def unplanned(dtype, seed, turn=0):
    """Single tokens, a prefix long enough for the wide kernel (4.8e9 operations)."""
    lens = [4610 + 1 + (11 * i) % 400 for i in range(128)]
    lens[5] = 0
    return ar.make(dtype, "planes", 16, 1, 32, 64, lens=lens[turn:] + lens[:turn], prefix=4610, layers=1, layer=0,
                   seed=seed)


def prompts(dtype, seed, turn=0):
    """Prompts and a draft: the wide kernel writes some results itself."""
    del turn  # starts and lengths belong together
    return ar.make(dtype, "planes", 16, 2, 4, 64, lens=[700, 650, 1300, 777], qlens=[130, 5, 99, 160], prefix=600,
                   layers=1, layer=0, seed=seed, room=ROOM)


CALLS = [planned, unplanned, prompts]


class Inputs:
    """Another case's device inputs, to be copied over a Run's on a stream."""

    def __init__(self, r, c):
        d = ar.Run(c)
        assert d.pool.shape == r.pool.shape and d.tables.shape == r.tables.shape
        self.c = c
        self.pairs = [(getattr(r, n), getattr(d, n).clone()) for n in
                      ("pool", "q", "tables", "prefix_pages", "lens", "q_start")]

    def load(self):
        for to, x in self.pairs:
            to.copy_(x)


def wanted(c):
    return ar.reference(c)


def near(got, want):
    out, lse = got
    o, l, tol, tol_l = want
    ar._near(out, o, tol, "out")
    ar._near(lse, l, tol_l, "lse")


@pytest.mark.parametrize("dtype", ["bf16", "fp8"])
@pytest.mark.parametrize("make", CALLS)
def test_replays_with_other_inputs(make, dtype):
    """A graph of two calls over one workspace, replayed on other lengths, tables, queries and pools."""
    first = make(dtype, 1)
    r = ar.Run(first)
    inputs = [Inputs(r, c) for c in (first, make(dtype, 2, 3), make(dtype, 3, 8))]
    want = [wanted(x.c) for x in inputs]
    other = torch.zeros_like(r.out)  # the first call's results, kept from the second
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        r.call()
        s.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            r.call()
            other.copy_(r.out)
            r.out.zero_()
            r.call()
    for k in (1, 0, 2, 0, 0, 1):
        with torch.cuda.stream(s):  # the copies end right in front of the replay
            inputs[k].load()
            g.replay()
        near(r.results(), want[k])
        assert torch.equal(other, r.out)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_streams_of_their_own(dtype):
    """Calls of every kind on streams of their own, with workspaces of their own, at once."""
    cases = [m(dtype, i) for i, m in enumerate(CALLS)]
    runs = [ar.Run(c) for c in cases]
    streams = [torch.cuda.Stream() for _ in runs]
    torch.cuda.synchronize()
    for _ in range(8):
        for r, s in zip(runs, streams):
            r.call(stream=s)
    torch.cuda.synchronize()
    for c, r in zip(cases, runs):
        near(r.results(), wanted(c))


@pytest.mark.parametrize("dtype", ["bf16", "fp8"])
@pytest.mark.parametrize("make", CALLS)
def test_call_behind_call(make, dtype):
    """Twelve calls over one workspace with nothing between them but the copies of the next inputs."""
    first = make(dtype, 4)
    r = ar.Run(first)
    inputs = [Inputs(r, first), Inputs(r, make(dtype, 5, 11))]
    want = [wanted(x.c) for x in inputs]
    r.ws.random_(0, 255)  # whatever the workspace holds
    r.ws[r.ws_bytes:] = 255
    torch.cuda.synchronize()
    got = []
    for i in range(12):
        inputs[i % 2].load()
        r.call()
        got.append((r.out.clone(), r.lse.clone()))
    r.results()
    for i, (out, lse) in enumerate(got):
        near((out.double().cpu(), lse.double().cpu()), want[i % 2])
