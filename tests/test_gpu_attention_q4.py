"""kvx.shared_attention over 4-bit pools against the definition in 64 bits."""
import math

import numpy as np
import pytest
import torch

from tests import attention_q4_ref as q4
from tests import quant_ref as qr

pytestmark = pytest.mark.gpu

KINDS = ["planes", "slots", "hnd"]


def run(c, **more):
    r = q4.Run(c)
    q4.check(c, r.call(**more).results())
    return r


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("H", [1, 2, 8])
def test_types_and_layouts(dtype, kind, D, H):
    run(q4.make(dtype, kind, 16, H, G=4, D=D, lens=[100, 37, 64, 33], prefix=32, seed=D))


@pytest.mark.parametrize("page", [1, 3, 16, 24, 64, 128, 1000])
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("D", [64, 128])
def test_page_sizes(page, kind, D):
    run(q4.make("bf16", kind, page, 1, G=5, D=D, lens=[211, 97, 130], prefix=77, seed=page))


@pytest.mark.parametrize("D", [32, 96, 160, 192, 256])
def test_head_dims(D):
    run(q4.make("bf16", "planes", 8, 2, G=3, D=D, lens=[50, 21], prefix=20, seed=D))


@pytest.mark.parametrize("G", [1, 2, 3, 7, 8, 9, 16, 17, 33, 65])
@pytest.mark.parametrize("H,D", [(1, 128), (3, 64), (5, 128)])
def test_head_counts(G, H, D):
    run(q4.make("bf16", "planes", 16, H, G=G, D=D, lens=[90, 70, 65], prefix=60, seed=G))


@pytest.mark.parametrize("H", [3, 5, 6, 9, 10, 16, 33])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("kind,page", [("planes", 16), ("slots", 1), ("hnd", 32), ("planes", 3), ("hnd", 8)])
def test_heads_that_share_a_cta(H, D, kind, page):
    """Chunks of heads that do not fill their places, or the last of which is smaller; every way of copying."""
    run(q4.make("bf16", kind, page, H, G=2, D=D, lens=[150, 33, 70], prefix=17, seed=H, layers=1, layer=0))


@pytest.mark.parametrize("H", [1, 2, 4, 8])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("kind,page", [("planes", 16), ("slots", 1), ("hnd", 64), ("planes", 1), ("slots", 24)])
@pytest.mark.parametrize("qlens", [None, (3, 9, 1, 33)])
def test_splits_of_rows_and_keys(H, D, kind, page, qlens):
    """Long enough for several stages of a CTA and pieces that go on; rows that take one to eight warps."""
    run(q4.make("f16", kind, page, H, G=3, D=D, lens=[2100, 333, 40, 1200], qlens=qlens, prefix=35, seed=H, layers=1,
                layer=0))


@pytest.mark.parametrize("n", [2500, 4100])
def test_many_tiny_requests(n):
    """More pieces a CTA than it lists at a time."""
    lens = [(i * 7) % 4 for i in range(n)]
    run(q4.make("bf16", "hnd", 16, 40, G=1, D=64, lens=lens, prefix=0, layers=1, layer=0))


@pytest.mark.parametrize("n", [1, 2, 15, 16, 17, 31, 32, 63, 64, 65, 127, 128, 129, 255, 256, 257, 700, 5000])
@pytest.mark.parametrize("prefix", [0, 1])
def test_lengths(n, prefix):
    run(q4.make("f16", "planes", 16, 1, G=4, D=128 if n % 2 else 64, lens=[n], prefix=(n - 1) * prefix, seed=n))


@pytest.mark.parametrize("D", [64, 96, 128])
def test_empty_rows_and_short_requests(D):
    run(q4.make("bf16", "planes", 16, 2, G=4, D=D, lens=[0, 300, 5, 200, 0, 1, 201, 64], prefix=200))


def test_nothing_at_all():
    run(q4.make("bf16", lens=[0, 0], prefix=0))
    run(q4.make("bf16", lens=[0, 0], prefix=40))


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("qlens", [(1, 8, 3, 5), (2, 2, 2, 2), (40, 1, 17, 90)])
def test_several_query_tokens(dtype, D, qlens):
    lens = [150 + q for q in qlens]
    lens[1] = 130 + qlens[1] - 1
    run(q4.make(dtype, "planes", 16, 2, G=4, D=D, lens=lens, qlens=qlens, prefix=130, seed=7))


@pytest.mark.parametrize("prefix", [0, 48, 250])
def test_more_queries_than_positions(prefix):
    run(q4.make("bf16", "planes", 16, 1, G=4, D=64, lens=[3, 0, 100, 20, 260], qlens=[6, 2, 100, 40, 300],
                prefix=prefix))


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("G", [4, 7])
def test_many_requests(D, G):
    lens = [1000 + 1 + 13 * (i % 9) for i in range(90)]
    run(q4.make("bf16", "planes", 16, 2, G=G, D=D, lens=lens, prefix=1000, layers=1, layer=0))


# With query starts the tables' room stands for the keys, so that small cases take the kernels of large ones.
ROOM = 300_000


@pytest.mark.parametrize("kind,page", [("planes", 1), ("planes", 4), ("slots", 8), ("hnd", 16), ("planes", 24),
                                       ("slots", 64), ("hnd", 128), ("hnd", 3)])
@pytest.mark.parametrize("prefix", [384, 517])
@pytest.mark.parametrize("D", [64, 128])
def test_wide_prefix_by_page_size(kind, page, prefix, D):
    lens = [prefix + 1 + 29 * (i % 5) for i in range(40)]
    run(q4.make("bf16", kind, page, 2, G=4, D=D, lens=lens, prefix=prefix, seed=page, room=ROOM, starts=True))


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("kind,page,prefix", [("planes", 16, 300), ("hnd", 32, 512), ("slots", 2, 260), ("planes", 64, 0)])
@pytest.mark.parametrize("D", [64, 128])
def test_prompts(dtype, kind, page, prefix, D):
    q = [200, 1, 77, 150]
    run(q4.make(dtype, kind, page, 2, G=4, D=D, lens=[prefix + 200, prefix + 50, prefix + 377, prefix + 150],
                qlens=q, prefix=prefix, seed=page, room=ROOM))


def test_prompts_among_padding_and_single_tokens():
    run(q4.make("f16", "planes", 16, 2, G=8, D=64, lens=[0, 700, 301, 0, 640, 333, 299],
                qlens=[1, 300, 1, 40, 5, 33, 60], prefix=300, room=ROOM))


def _spread_scales(D):
    """Values' groups multiplied by powers of two that lie far apart."""
    def edit(b):
        pair = b[..., D // 2:].view(np.float16)
        g = np.random.default_rng(b.size)
        f = g.choice([2.0 ** -8, 1, 1, 2.0 ** 6], size=pair.shape[-1] // 2)
        pair[:, 1, :, 0::2] = pair[:, 1, :, 0::2] * f
        pair[:, 1, :, 1::2] = pair[:, 1, :, 1::2] * f
    return edit


@pytest.mark.parametrize("D", [64, 96, 128])
def test_values_far_from_zero_and_of_every_size(D):
    """Lows far greater than the scales; groups whose scales lie far apart; large and tiny values."""
    run(q4.make("bf16", "planes", 16, 2, G=4, D=D, lens=[500, 300, 411], prefix=100, shift=5.0,
                edit_bytes=_spread_scales(D)))


@pytest.mark.parametrize("D", [64, 128])
def test_the_same_with_many_rows(D):
    run(q4.make("bf16", "planes", 16, 2, G=4, D=D, lens=[500, 300, 411], qlens=[70, 40, 90], prefix=100, shift=5.0,
                edit_bytes=_spread_scales(D), room=ROOM))


def _pairs(b, D):
    """(scales, lows) of tokens' bytes [tokens, 2, H, bytes], to be changed in place."""
    pair = b[..., D // 2:].view(np.float16)
    return pair[..., 0::2], pair[..., 1::2]


def _falling(D):
    """Scales below 0, as a quantiser of another convention may have them: elements fall as codes rise."""
    def edit(b):
        scale, low = _pairs(b, D)
        top = (low.astype(np.float32) + 15 * scale.astype(np.float32)).astype(np.float16)
        scale[:], low[:] = -scale * np.float16(32), top * np.float16(32)
    return edit


@pytest.mark.parametrize("D,qlens", [(64, None), (96, None), (128, None), (64, [70, 40]), (128, [70, 40])])
def test_scales_below_0(D, qlens):
    """32 times the usual values, so that weights as they are would not fit next to such a scale."""
    run(q4.make("bf16", "planes", 16, 2, G=4, D=D, lens=[500, 300], qlens=qlens, prefix=100, scale=1e-3,
                edit_bytes=_falling(D), room=ROOM))


def _far_keys(D):
    """Keys from -61440 to 61440, groups whose codes times their scale pass f16's end among them."""
    def edit(b):
        scale, low = (x[:, 0] for x in _pairs(b, D))
        lows = np.clip(low.astype(np.float32) * 2.0 ** 13.4, -61440, 0).astype(np.float16)
        most = (61440 - lows.astype(np.float32)) / 15
        scale[:] = np.minimum(scale.astype(np.float32) * 2.0 ** 13.4, most * (1 - 2.0 ** -10)).astype(np.float16)
        low[:] = lows
        assert (scale > 4400).any() and (scale < 3900).any()
    return edit


@pytest.mark.parametrize("D,qlens", [(64, None), (128, None), (64, [70, 40]), (128, [70, 40])])
def test_keys_at_the_ends_of_the_range(D, qlens):
    run(q4.make("bf16", "planes", 16, 2, G=4, D=D, lens=[500, 300], qlens=qlens, prefix=100, scale=2.0 ** -18,
                edit_bytes=_far_keys(D), room=ROOM))


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("what", [0x7C00, 0xFC00, 0x7E00])
def test_prompts_mask_infinities_and_nan(D, what):
    """The last tokens of a prompt of many rows, as below; with lows of infinity alone too."""
    c = q4.make("bf16", "planes", 16, 1, G=2, D=D, lens=[270], qlens=[200], prefix=0, layers=1, layer=0, room=2 * ROOM)
    pool = c.pool.view(2, c.slots, D // 8 * 5)
    for j in (266, 267, 269):
        slot = int(c.tables[0, j // 16]) * 16 + j % 16
        pool[:, slot, D // 2:] = torch.tensor([what & 255, what >> 8] * (D // 16), dtype=torch.uint8)
    out, lse = q4.Run(c).call().results()
    want, wlse, tol, tol_l = q4.reference(c)
    q4.ar._near(out[:196], want[:196], tol[:196], "out")
    q4.ar._near(lse[:196], wlse[:196], tol_l[:196], "lse")
    assert not bool(torch.isfinite(out[196:]).any())


@pytest.mark.parametrize("D", [64, 128])
def test_scales_that_grow_along_the_keys(D):
    """The greatest scale of the values comes late: what was summed before keeps its share."""
    def edit(b):
        pair = b[..., D // 2:].view(np.float16)
        up = 2.0 ** np.linspace(-10, 12, len(b)).round()
        pair[:, 1] = (pair[:, 1].astype(np.float64) * up[:, None, None]).astype(np.float16)
    run(q4.make("bf16", "planes", 16, 1, G=3, D=D, lens=[900], prefix=0, edit_bytes=edit))


@pytest.mark.parametrize("D", [64, 96, 128])
@pytest.mark.parametrize("what", [0x7C00, 0xFC00, 0x7E00])
def test_masked_keys_hold_infinities_and_nan(D, what):
    """The last tokens' scales and lows are not finite: rows that do not see them are untouched."""
    c = q4.make("bf16", "planes", 16, 1, G=2, D=D, lens=[70], qlens=[6], prefix=0, layers=1, layer=0)
    size = D // 8 * 5
    pool = c.pool.view(2, c.slots, size)
    for j in (67, 68, 69):
        slot = int(c.tables[0, j // 16]) * 16 + j % 16
        pool[:, slot, D // 2:] = torch.tensor([what & 255, what >> 8] * (D // 16), dtype=torch.uint8)
    r = q4.Run(c)
    out, lse = r.call().results()
    want, wlse, tol, tol_l = q4.reference(c)
    q4.ar._near(out[:3], want[:3], tol[:3], "out")
    q4.ar._near(lse[:3], wlse[:3], tol_l[:3], "lse")
    assert not bool(torch.isfinite(out[3:]).any())


def test_infinite_values_reach_the_rows_that_see_them():
    """A value's low of infinity: its weight is positive, so its columns are infinite, the others as ever."""
    c = q4.make("bf16", "planes", 16, 1, G=4, D=128, lens=[80], prefix=0, layers=1, layer=0)
    slot = int(c.tables[0, 2]) * 16 + 5
    pool = c.pool.view(2, c.slots, 80)
    pool[1, slot, 64 + 4 * 2 + 2:64 + 4 * 2 + 4] = torch.tensor([0, 0x7C], dtype=torch.uint8)  # low of group 2
    c.kv[0][37, 1, 0, 64:96], c.mag[0][37, 1, 0, 64:96] = math.inf, math.inf
    out, lse = q4.Run(c).call().results()
    want, _, tol, _ = q4.reference(c)
    assert bool((out[..., 64:96] == math.inf).all())
    keep = [i for i in range(128) if not 64 <= i < 96]
    q4.ar._near(out[..., keep], want[..., keep], tol[..., keep], "out")


@pytest.mark.parametrize("k_scale,v_scale,scale", [(0.5, 3.0, None), (-1.0, 2.0, None), (1.0, 1.0, 0.0), (1.0, -1.0, 2.0)])
def test_scales(k_scale, v_scale, scale):
    run(q4.make("bf16", "planes", 16, 2, G=4, D=128, lens=[100, 61], prefix=30, k_scale=k_scale, v_scale=v_scale,
                scale=scale, spread=0.5))


@pytest.mark.parametrize("kind,offset,pad", [("planes", 4, 0), ("planes", 0, 4), ("slots", 8, 12), ("planes", 16, 16)])
@pytest.mark.parametrize("D", [64, 128])
def test_pools_off_16_bytes(kind, offset, pad, D):
    run(q4.make("bf16", kind, 16, 2, G=4, D=D, lens=[100, 61], prefix=30, offset=offset, slot_pad=pad))


def test_same_call_same_bits():
    c = q4.make("bf16", "planes", 16, 2, G=4, D=128, lens=[3000, 61, 900], prefix=30)
    r = q4.Run(c)
    first = [x.clone() for x in r.call().results()]
    for _ in range(3):
        for a, b in zip(first, r.call().results()):
            assert torch.equal(a, b)


def test_large_queries():
    """bf16 queries past f16's range."""
    c = q4.make("bf16", "planes", 16, 2, G=4, D=128, lens=[200, 61], prefix=30, spread=1e6, scale=1e-7)
    run(c)
    run(q4.make("bf16", "planes", 16, 2, G=4, D=64, lens=[200, 61], prefix=30, spread=1e-6, scale=1e5))


@pytest.mark.parametrize("kind,page,D", [("planes", 16, 128), ("slots", 1, 128), ("planes", 3, 128), ("hnd", 16, 64),
                                         ("hnd", 3, 128), ("planes", 16, 96)])
def test_a_bad_page_is_reported(kind, page, D):
    c = q4.make("bf16", kind, page, 2, G=4, D=D, lens=[200, 61], prefix=30)
    for bad in (c.pages, -1, 2 ** 31 - 1):
        r = q4.Run(c)
        r.tables[0, 150 // page] = bad
        r.call()
        torch.cuda.synchronize()
        assert int(r.status.item()) == r.kvx.ERR_OUT_OF_RANGE


def test_captured_and_replayed():
    c = q4.make("bf16", "planes", 16, 2, G=4, D=128, lens=[300, 61, 144], prefix=130)
    r = q4.Run(c)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        r.call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        r.call()
    for seed in (1, 2):
        d = q4.make("bf16", "planes", 16, 2, G=4, D=128, lens=[300, 61, 144], prefix=130, seed=seed)
        r.pool.copy_(d.pool)
        r.q.copy_(d.q)
        r.tables.copy_(d.tables)
        r.prefix_pages.copy_(d.prefix_pages)
        graph.replay()
        q4.check(d, r.results())


def test_tokens_of_no_request():
    """Query tokens behind the last request's get 0 and -infinity."""
    c = q4.make("bf16", "planes", 16, 2, G=4, D=128, lens=[60, 61], qlens=[2, 3], prefix=20)
    r = q4.Run(c, extra_tokens=3)
    out, lse = r.call().results()
    q4.check(c, (out, lse))
    assert bool((out[c.T:] == 0).all() and (lse[c.T:] == -math.inf).all())


@pytest.mark.parametrize("kind,page", [("planes", 16), ("planes", 1), ("hnd", 16)])
def test_planes_past_4_gib(kind, page):
    """Pages whose bytes begin beyond 2^32 of a plane."""
    from disaggregated_paged_kv_gb300 import kvx
    H, D, S = 8, 128, 80
    slots = 16 * 450_000
    pool = torch.full((2 * slots * H * S,), 255, dtype=torch.uint8, device="cuda")
    more = dict(kind=kvx.HND_PAGED, page_size=page) if kind == "hnd" else {}
    layout = kvx.Layout(1, H, D, kvx.Q4, slots, base=pool, plane_stride=slots * H * S, **more)
    c = q4.make("bf16", kind, page, H, G=4, D=D, lens=[100], prefix=0, layers=1, layer=0)
    n = -(-100 // page)
    far = torch.arange(n, dtype=torch.int32) + slots // page - n - 3
    small, big = c.pool.view(2, -1, page * H * S), pool.view(2, -1, page * H * S)
    for j in range(n):
        big[:, int(far[j])] = small[:, int(c.tables[0, j])].cuda()
    r = q4.Run(c)
    r.layout = layout
    r.tables[0, :n] = far.cuda()
    q4.check(c, r.call().results())


def test_one_page_beyond_31_bits_of_words():
    """A head-major pool that is a single page of more than 2^31 8-byte words a head: all its keys are zeros but the
    last 40 (scores 0, values 0), so that the sums are known."""
    from disaggregated_paged_kv_gb300 import kvx
    D, S, G, last = 128, 80, 4, 40
    slots = (2 ** 31 // 10 + 1000) // 16 * 16
    pool = torch.zeros(2, slots, S, dtype=torch.uint8, device="cuda")
    layout = kvx.Layout(1, 1, D, kvx.Q4, slots, base=pool, plane_stride=slots * S, kind=kvx.HND_PAGED, page_size=slots)
    g = np.random.default_rng(0)
    held = qr.encode_q4(g.standard_normal((last, 2, 1, D)).astype(np.float32) * 8, 1.0)
    pool[:, -last:] = torch.from_numpy(held)[:, :, 0].transpose(0, 1).cuda()
    code, step, low = qr.parts_q4(held, D)
    k, v = torch.from_numpy(code * step + low).double()[:, :, 0].unbind(1)
    q = (torch.from_numpy(g.standard_normal((1, G, D))) * 2).half().cuda()
    out, lse = torch.full_like(q, math.nan), torch.full((1, G), math.nan, device="cuda")
    ws = torch.empty(kvx.attention_workspace_size(layout, 1, 1, G, 0), dtype=torch.uint8, device="cuda")
    status = torch.full((1,), -1, dtype=torch.int32, device="cuda")
    kvx.shared_attention(layout, 0, q, out, torch.zeros(1, 1, dtype=torch.int32, device="cuda"),
                         torch.tensor([slots], dtype=torch.int32, device="cuda"), slots, ws, status, lse=lse)
    torch.cuda.synchronize()
    assert status.item() == kvx.OK
    s = q.cpu().double()[0] @ k.T * D ** -0.5
    most = s.max(1).values.clamp(min=0)
    l = (slots - last) * (-most).exp() + (s - most[:, None]).exp().sum(1)
    want = ((s - most[:, None]).exp() @ v) / l[:, None]
    # beside the rounding of a weight, of its product with a scale and of the result (2^-11 each; v is up to 2^5, the
    # lows' part up to as much again): the sum of 2^28 equal weights, split 2432 ways or more and over 8 rows of keys, takes
    # no more than 2^13 additions in a row, each off by 2^-24
    weight = ((s - most[:, None]).exp() @ v.abs()) / l[:, None]
    assert bool(((out.cpu().double()[0] - want).abs() <= 2 ** -11 * want.abs() + (2 ** -8 + 2 ** -11) * weight + 2 ** -24).all())
    assert bool((lse.cpu().double()[0] - (l.log() + most)).abs().max() <= 2 ** -11 + 2 ** -16)


def test_two_calls_at_once():
    """Two streams, workspaces of their own."""
    runs = [q4.Run(q4.make("bf16", "planes", 16, 8, G=4, D=128, lens=[900 + i, 61, 300], prefix=30, seed=i, layers=1, layer=0))
            for i in range(2)]
    streams = [torch.cuda.Stream() for _ in runs]
    torch.cuda.synchronize()
    for _ in range(3):
        for r, s in zip(runs, streams):
            r.call(stream=s)
    torch.cuda.synchronize()
    for r in runs:
        q4.check(r.c, r.results())
