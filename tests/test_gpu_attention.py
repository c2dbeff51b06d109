"""kvx.shared_attention against the definition in 64 bits: types, layouts, lengths from nothing to
many tiles, masks that fall inside tiles, garbage in masked places, and refusals."""
import math

import pytest
import torch

from tests import attention_ref as ar

pytestmark = pytest.mark.gpu

TYPES = ["bf16", "f16", "fp8", "f32"]
KINDS = ["planes", "slots", "hnd"]


def run(c, **more):
    r = ar.Run(c)
    ar.check(c, r.call(**more).results())
    return r


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("D", [64, 128])
def test_types_and_layouts(dtype, kind, D):
    run(ar.make(dtype, kind, 16, 2, 4, D, lens=[100, 37, 64, 33], prefix=32, seed=D))


@pytest.mark.parametrize("page", [1, 3, 16, 24, 64, 128, 1000])
@pytest.mark.parametrize("kind", KINDS)
def test_page_sizes(page, kind):
    run(ar.make("bf16", kind, page, 1, 5, 128, lens=[211, 97, 130], prefix=77, seed=page))


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("D", [1, 7, 8, 16, 48, 80, 96, 129, 192, 256])
def test_head_dims(dtype, D):
    run(ar.make(dtype, "planes", 8, 2, 3, D, lens=[50, 21], prefix=20, seed=D))


@pytest.mark.parametrize("G", [1, 2, 3, 7, 8, 16, 17, 33])
@pytest.mark.parametrize("H", [1, 3])
def test_head_counts(G, H):
    run(ar.make("bf16", "planes", 16, H, G, 64, lens=[90, 70, 65], prefix=60, seed=G))


@pytest.mark.parametrize("n", [1, 2, 15, 16, 17, 31, 32, 63, 64, 65, 127, 128, 129, 255, 256, 257, 700, 5000])
@pytest.mark.parametrize("prefix", [0, 1])
def test_lengths(n, prefix):
    """One request from a single token up; prefix 1: all of it but a token's worth is shared."""
    run(ar.make("f16", "planes", 16, 1, 4, 64, lens=[n], prefix=(n - 1) * prefix, seed=n))


@pytest.mark.parametrize("dtype", ["bf16", "fp8", "f32"])
def test_empty_rows_and_short_requests(dtype):
    """Padding rows, requests shorter than the prefix, and one that is the prefix exactly."""
    run(ar.make(dtype, "planes", 16, 2, 4, 128, lens=[0, 300, 5, 200, 0, 1, 201, 64], prefix=200))


def test_nothing_at_all():
    run(ar.make("bf16", lens=[0, 0], prefix=0))
    run(ar.make("bf16", lens=[0, 0], prefix=40))
    r = ar.Run(ar.make("bf16", lens=[], prefix=0))
    r.call().results()


@pytest.mark.parametrize("dtype", ["bf16", "f16", "fp8", "f32"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("qlens", [(1, 8, 3, 5), (2, 2, 2, 2), (40, 1, 17, 90)])
def test_several_query_tokens(dtype, D, qlens):
    lens = [150 + q for q in qlens]
    lens[1] = 130 + qlens[1] - 1
    run(ar.make(dtype, "planes", 16, 2, 4, D, lens=lens, qlens=qlens, prefix=130, seed=7))


@pytest.mark.parametrize("prefix", [0, 48, 250])
def test_more_queries_than_positions(prefix):
    """The first query tokens see nothing, or less than the prefix."""
    run(ar.make("bf16", "planes", 16, 1, 4, 64, lens=[3, 0, 100, 20, 260], qlens=[6, 2, 100, 40, 300],
                prefix=prefix))


def test_requests_without_query_tokens():
    run(ar.make("bf16", "planes", 16, 2, 4, 64, lens=[80, 90, 100], qlens=[0, 3, 0], prefix=64))


@pytest.mark.parametrize("dtype", ["bf16", "f16", "fp8"])
@pytest.mark.parametrize("G", [4, 7])
def test_prompt(dtype, G):
    """Hundreds of rows of one request, behind a prefix of several hundred tokens."""
    run(ar.make(dtype, "hnd", 16, 2, G, 128, lens=[500 + 333, 500 + 100], qlens=[333, 100],
                prefix=500))


@pytest.mark.parametrize("dtype", ["bf16", "f16", "fp8"])
@pytest.mark.parametrize("D", [64, 128])
def test_many_requests(dtype, D):
    """Enough rows for whole tiles of them over the prefix, more keys than a split has."""
    lens = [1000 + 1 + 13 * (i % 9) for i in range(90)]
    run(ar.make(dtype, "planes", 16, 2, 7, D, lens=lens, prefix=1000, layers=1, layer=0))


@pytest.mark.parametrize("dtype", ["bf16", "f16", "fp8"])
@pytest.mark.parametrize("kind,page", [("planes", 1), ("planes", 4), ("slots", 8), ("hnd", 16),
                                       ("planes", 24), ("slots", 64), ("hnd", 128), ("hnd", 3)])
@pytest.mark.parametrize("prefix", [384, 517])
def test_many_rows_by_page_size(dtype, kind, page, prefix):
    """Tiles of many rows over whole pages, parts of pages, and a prefix that ends inside one."""
    lens = [prefix + 1 + 29 * (i % 5) for i in range(40)]
    run(ar.make(dtype, kind, page, 2, 4, 64 if page == 8 else 128, lens=lens, prefix=prefix,
                layers=2, layer=1, seed=page))


@pytest.mark.parametrize("dtype", ["bf16", "fp8"])
@pytest.mark.parametrize("kind,page,prefix", [("planes", 16, 300), ("hnd", 32, 512), ("slots", 2, 260),
                                              ("planes", 64, 0)])
def test_prompts_by_page_size(dtype, kind, page, prefix):
    """Prompts walk from the prefix's pages into their own inside a tile of keys."""
    q = [200, 1, 77, 150]
    run(ar.make(dtype, kind, page, 2, 4, 128, lens=[prefix + 200, prefix + 50, prefix + 377, prefix + 150],
                qlens=q, prefix=prefix, seed=page))


def test_prompts_among_padding_and_single_tokens():
    run(ar.make("f16", "planes", 16, 2, 8, 64, lens=[0, 700, 301, 0, 640, 333, 299],
                qlens=[1, 300, 1, 40, 5, 33, 60], prefix=300))


# Calls of many rows go to the kernel of 128-row tiles from some 4.5e9 operations on.  With query starts the
# tables' room stands for the keys, so that small cases get there; without, the prefix has to be that long.
ROOM = 300_000


@pytest.mark.parametrize("dtype", ["bf16", "f16", "fp8"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("G", [1, 4, 7])
def test_wide_prefix(dtype, D, G):
    lens = [1000 + 1 + 13 * (i % 9) for i in range(90)]
    run(ar.make(dtype, "planes", 16, 2, G, D, lens=lens, prefix=1000, layers=1, layer=0, room=ROOM,
                starts=True))


@pytest.mark.parametrize("dtype", ["bf16", "f16", "fp8"])
@pytest.mark.parametrize("kind,page", [("planes", 1), ("planes", 4), ("slots", 8), ("hnd", 16),
                                       ("planes", 24), ("slots", 64), ("hnd", 128), ("hnd", 3)])
@pytest.mark.parametrize("prefix", [384, 517])
def test_wide_by_page_size(dtype, kind, page, prefix):
    lens = [prefix + 1 + 29 * (i % 5) for i in range(40)]
    run(ar.make(dtype, kind, page, 2, 4, 64 if page == 8 else 128, lens=lens, prefix=prefix,
                layers=2, layer=1, seed=page, room=ROOM, starts=True))


@pytest.mark.parametrize("dtype", ["bf16", "f16", "fp8"])
@pytest.mark.parametrize("kind,page,prefix", [("planes", 16, 300), ("hnd", 32, 512), ("slots", 2, 260),
                                              ("planes", 64, 0)])
@pytest.mark.parametrize("G", [4, 7])
def test_wide_prompts(dtype, kind, page, prefix, G):
    run(ar.make(dtype, kind, page, 2, G, 128, lens=[prefix + 200, prefix + 50, prefix + 377, prefix + 150],
                qlens=[200, 1, 77, 150], prefix=prefix, seed=page, room=ROOM))


@pytest.mark.parametrize("dtype", ["bf16", "fp8"])
@pytest.mark.parametrize("D", [64, 128])
def test_wide_with_padding_short_and_single(dtype, D):
    run(ar.make(dtype, "planes", 16, 2, 8, D, lens=[0, 700, 301, 0, 640, 333, 299, 20, 300],
                qlens=[1, 300, 1, 40, 5, 33, 60, 20, 1], prefix=300, room=ROOM))
    run(ar.make(dtype, "planes", 16, 1, 4, D, lens=[3, 0, 100, 20, 260], qlens=[6, 2, 100, 40, 300],
                prefix=250, room=ROOM))
    run(ar.make(dtype, "planes", 16, 2, 4, D, lens=[0] * 30 + [260, 5, 256, 90] * 6, prefix=256, room=ROOM,
                starts=True))


@pytest.mark.parametrize("dtype", ["bf16", "f16", "fp8"])
def test_wide_sharp_and_rising_scores(dtype):
    run(ar.make(dtype, "planes", 16, 2, 8, 64, lens=[700, 650], qlens=[150, 100], prefix=390, spread=30.0,
                room=ROOM))

    def edit(c):
        c.q[:] = 1.0
        for x in [c.common] + c.kv:
            x[:, 0] = ((torch.arange(len(x)) / 4.0).to(x.dtype))[:, None, None]
    run(ar.make(dtype, "planes", 16, 1, 4, 64, lens=[600], qlens=[90], prefix=0, edit=edit, room=ROOM,
                k_scale=1.0))


@pytest.mark.parametrize("dtype", ["bf16", "f16", "fp8"])
@pytest.mark.parametrize("value", [math.nan, math.inf, -math.inf])
def test_wide_garbage_behind_the_mask(dtype, value):
    """As test_garbage_behind_the_mask, in tiles of 128 rows."""
    if dtype == "fp8" and not math.isnan(value):
        pytest.skip("E4M3 has no infinities")

    def edit(c):
        c.kv[0][c.lens[0] - 150:, 1] = torch.tensor(value).to(c.kv[0].dtype)
        c.kv[1][c.lens[1] - 1:, 0] = torch.tensor(value).to(c.kv[1].dtype)
    c = ar.make(dtype, "planes", 16, 1, 4, 64, lens=[230, 140, 29], qlens=[200, 90, 1], prefix=20, edit=edit,
                room=ROOM)
    out, lse = ar.Run(c).call().results()
    want, wlse, tol, tol_l = ar.reference(c)
    sees = torch.zeros(c.T, dtype=torch.bool)
    sees[c.start[1] - 150:c.start[1]] = True       # V
    last = torch.zeros_like(sees)
    last[c.start[2] - 1] = True                    # K
    ok = ~sees & ~last
    assert bool(((out - want).abs()[ok] <= tol[ok]).all())
    assert bool(((lse - wlse).abs()[~last] <= tol_l[~last]).all())
    assert not bool(torch.isfinite(out[sees]).any())


@pytest.mark.parametrize("dtype", ["bf16", "fp8"])
def test_wide_garbage_in_the_prefix(dtype):
    """Prefix positions that some requests do not reach hold NaN values."""
    def edit(c):
        for x in [c.common] + c.kv:
            x[300:, 1] = torch.tensor(math.nan).to(x.dtype)
    c = ar.make(dtype, "planes", 16, 1, 4, 64, lens=[290, 300, 301, 600] * 10, prefix=500, edit=edit,
                room=ROOM, starts=True)
    out, lse = ar.Run(c).call().results()
    want, wlse, tol, tol_l = ar.reference(c)
    for i, n in enumerate(c.lens):
        if n <= 300:
            assert bool(((out - want).abs()[i] <= tol[i]).all())
        else:
            assert bool(torch.isnan(out[i]).all())
    assert bool(((lse - wlse).abs() <= tol_l).all())


@pytest.mark.parametrize("dtype,kind", [("bf16", "planes"), ("f16", "hnd"), ("fp8", "slots")])
@pytest.mark.parametrize("own", [3, 700])
def test_wide_decode_step(dtype, kind, own):
    """Single tokens without query starts, a prefix long enough for the wide kernel."""
    lens = [4610 + 1 + (own * i) % (2 * own) for i in range(128)]
    lens[5] = 0
    lens[77] = 4000
    run(ar.make(dtype, kind, 16, 1, 32, 64, lens=lens, prefix=4610, layers=1, layer=0))


@pytest.mark.parametrize("scale", [-0.125, 0.0])
def test_scales_that_turn_scores_round(scale):
    run(ar.make("bf16", "planes", 16, 2, 4, 64, lens=[200 + i for i in range(40)], prefix=190, scale=scale,
                room=ROOM, starts=True))


def test_wide_queries_and_results_off_16_bytes():
    c = ar.make("bf16", "planes", 16, 1, 4, 64, lens=[300, 330], qlens=[60, 90], prefix=200, room=ROOM)
    r = ar.Run(c)
    wide = torch.empty(c.T, 4 * 64 + 11, dtype=torch.bfloat16, device="cuda")
    q = wide[:, 3:3 + 256].unflatten(1, (4, 64))
    q.copy_(r.q)
    r.q = q
    r.out = torch.empty_like(wide)[:, 1:1 + 256].unflatten(1, (4, 64))
    ar.check(c, r.call().results())


def test_wide_same_bits_again():
    c = ar.make("bf16", lens=[700, 650, 1300], qlens=[130, 5, 99], prefix=600, layers=1, layer=0, room=ROOM)
    r = ar.Run(c)
    a = r.call().results()
    r.out.fill_(0)
    r.ws.fill_(255)
    b = r.call().results()
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_wide_device_refusals():
    for edit, want in [
        (lambda r: r.lens.fill_(-1), "INVALID_ARG"),
        (lambda r: r.lens.fill_(2 ** 30), "OUT_OF_RANGE"),
        (lambda r: r.tables.fill_(-1), "OUT_OF_RANGE"),
        (lambda r: r.prefix_pages.fill_(2 ** 31 - 1), "OUT_OF_RANGE"),
    ]:
        for dtype in ("bf16", "fp8"):
            for kw in (dict(lens=[300 + i for i in range(70)], starts=True),
                       dict(lens=[400, 450], qlens=[100, 150])):
                r = ar.Run(ar.make(dtype, D=128, prefix=250, layers=1, layer=0, room=ROOM, **kw))
                edit(r)
                assert _status(r) == getattr(r.kvx, "ERR_" + want)


def test_offsets_past_32_bits():
    """Pages at the end of planes of over 4 GiB, in token rows, head-major pages and a slot-major pool."""
    kvx = ar.Run(ar.make("bf16", lens=[50])).kvx
    c = ar.make("bf16", "planes", 16, 2, 4, 128, lens=[300, 333] + [290 + i for i in range(20)], prefix=280,
                layers=1, layer=0)
    R = c.H * c.D * 2
    slots = (9 << 30) // (2 * R) // 16 * 16                    # two planes of 4.5 GiB
    far = slots // 16 - c.pages
    small = c.pool.view(torch.bfloat16).view(2, c.pages, 16, c.H, c.D).cuda()
    for kind in ("planes", "hnd", "slots"):
        pool = torch.empty(2 * slots * c.H * c.D, dtype=torch.bfloat16, device="cuda")
        if kind == "planes":
            pool.view(2, slots // 16, 16, c.H, c.D)[:, far:] = small
            more = dict(plane_stride=slots * R)
        elif kind == "hnd":
            pool.view(2, slots // 16, c.H, 16, c.D)[:, far:] = small.transpose(2, 3)
            more = dict(plane_stride=slots * R, kind=kvx.HND_PAGED, page_size=16)
        else:
            pool.view(slots // 16, 16, 2, c.H, c.D)[far:] = small.permute(1, 2, 0, 3, 4)
            more = dict(plane_stride=R, slot_stride=2 * R)
        for starts in (False, True):  # narrow kernel; with room in the tables the wide one too
            r = ar.Run(c)
            r.pool = None
            r.layout = kvx.Layout(1, c.H, c.D, kvx.BF16, slots, base=pool, keepalive=pool, **more)
            wide = torch.full((len(c.lens), 20000 if starts else c.tables.shape[1]), -1, dtype=torch.int32,
                              device="cuda")
            for b, n in enumerate(c.lens):
                k = -(-n // 16)
                wide[b, :k] = c.tables[b, :k].cuda() + far
            r.tables = wide
            r.prefix_pages = r.prefix_pages + far
            ar.check(c, r.call(q_start=r.q_start if starts else None).results())
            r.layout.close()
        del pool


@pytest.mark.parametrize("n", [1100, 2100])
@pytest.mark.parametrize("starts", [False, True])
def test_many_small_requests(n, starts):
    """More requests than the plan keeps at hand, and (single tokens) more than calls without one take."""
    run(ar.make("f16", "planes", 4, 1, 2, 64, lens=[(7 * i) % 23 for i in range(n)], prefix=6, layers=1,
                layer=0, starts=starts))


def test_more_kv_heads_than_multiprocessors():
    run(ar.make("bf16", "planes", 8, 160, 1, 64, lens=[40, 33, 90], prefix=24, layers=1, layer=0))
    run(ar.make("bf16", "planes", 8, 160, 2, 64, lens=[140, 133], qlens=[40, 37], prefix=24, layers=1,
                layer=0, room=20000))


def test_long_and_short_together():
    run(ar.make("bf16", "planes", 16, 1, 4, 128, lens=[9000, 1, 30, 4000], prefix=0, layers=1, layer=0))


@pytest.mark.parametrize("dtype", TYPES)
def test_sharp_scores(dtype):
    """Scores over a range of hundreds: most weights vanish, the running maximum rises and falls."""
    run(ar.make(dtype, "planes", 16, 2, 4, 64, lens=[400, 700, 650], prefix=390, spread=30.0))


def test_rising_scores():
    """Every key scores higher than the one before: the maximum is renewed throughout."""
    def edit(c):
        c.q[:] = 1.0
        for x in c.kv:
            x[:, 0] = (torch.arange(len(x)) / 4.0)[:, None, None]
    run(ar.make("f16", "planes", 16, 1, 4, 64, lens=[600], prefix=0, edit=edit))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_low_scores(dtype):
    """Scores near the type's lowest values stay ordinary rows."""
    def edit(c):
        c.q[:] = 1.0
        for x in c.kv:
            x[:, 0] = -1e36
        c.common[:, 0] = -1e36
    c = ar.make(dtype, "planes", 16, 1, 2, 16, lens=[50, 20], prefix=10, edit=edit)
    out, lse = ar.Run(c).call().results()
    want = torch.stack([x[:, 1].double().mean(0) for x in c.kv])  # equal scores
    assert torch.allclose(out, want.repeat_interleave(2, 1), rtol=0, atol=0.02)
    assert bool((lse < -1e36).all()) and bool(torch.isfinite(lse).all())


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("value", [math.nan, math.inf, -math.inf])
@pytest.mark.parametrize("n", [40, 200])
def test_garbage_behind_the_mask(dtype, value, n):
    """A draft's later tokens hold NaN or infinities: only the rows that see them may show it."""
    bad = 3 if n == 40 else 150
    def edit(c):
        c.kv[0][c.lens[0] - bad:, 1] = value
        c.kv[1][c.lens[1] - 1:, 0] = value
    c = ar.make(dtype, "planes", 16, 1, 4, 64, lens=[n + 30, n + 20, n + 9], qlens=[n, 4, 1],
                prefix=20, edit=edit)
    out, lse = ar.Run(c).call().results()
    want, wlse, tol, tol_l = ar.reference(c)
    sees = torch.zeros(c.T, dtype=torch.bool)
    sees[c.start[0] + n - bad:c.start[1]] = True   # V
    last = torch.zeros_like(sees)
    last[c.start[2] - 1] = True                    # K
    ok = ~sees & ~last
    assert bool(((out - want).abs()[ok] <= tol[ok]).all())
    assert bool(((lse - wlse).abs()[~last] <= tol_l[~last]).all())
    assert not bool(torch.isfinite(out[sees]).any())
    if math.isnan(value):
        assert bool(torch.isnan(out[last]).all())


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_garbage_beyond_a_short_request(dtype):
    """Prefix positions that a short request does not see hold NaN values."""
    def edit(c):
        c.common[100:, 1] = math.nan
        for b, n in enumerate(c.lens):
            c.kv[b][100:, 1] = math.nan
    c = ar.make(dtype, "planes", 16, 1, 4, 64, lens=[90, 100, 101, 300], prefix=200, edit=edit)
    out, lse = ar.Run(c).call().results()
    want, wlse, tol, tol_l = ar.reference(c)
    assert bool(((out - want).abs()[:2] <= tol[:2]).all())
    assert bool(torch.isnan(out[2:]).all())
    assert bool(((lse - wlse).abs() <= tol_l).all())


def test_minus_infinity_scores():
    """Keys of -inf score weigh nothing; a row that sees only those is empty."""
    def edit(c):
        c.q[:] = 1.0
        c.kv[0][:, 0] = -math.inf
        c.kv[1][5:, 0] = -math.inf
    c = ar.make("bf16", "planes", 16, 1, 4, 64, lens=[40, 40], prefix=0, edit=edit)
    out, lse = ar.Run(c).call().results()
    assert bool((out[0] == 0).all()) and bool((lse[0] == -math.inf).all())
    c.kv[1] = c.kv[1][:5]
    c.lens[1] = 5
    want, wlse, tol, tol_l = ar.reference(c)
    assert bool(((out - want).abs()[1] <= tol[1]).all())
    assert bool(((lse - wlse).abs()[1] <= tol_l[1]).all())


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("kind,offset,pad", [("planes", 1, 0), ("slots", 3, 0), ("slots", 0, 5),
                                             ("slots", 8, 24), ("hnd", 1, 0)])
def test_odd_addresses(dtype, kind, offset, pad):
    """Planes and slots that are only element aligned."""
    run(ar.make(dtype, kind, 8, 2, 4, 64, lens=[70, 33], prefix=30, offset=offset, slot_pad=pad))


def test_strided_output_and_no_lse():
    c = ar.make("bf16", lens=[50, 60], prefix=16)
    r = ar.Run(c, lse=False)
    got = r.call().results()
    ar.check(c, got)
    # the heads beside the written ones are untouched
    base = r.out._base if r.out._base is not None else r.out
    assert bool(torch.isnan(base[:, 0].float()).all()) and bool(torch.isnan(base[:, -1].float()).all())


def test_tokens_of_no_request():
    """Query tokens past the last request's end get nothing."""
    c = ar.make("bf16", lens=[80, 90], qlens=[3, 2], prefix=64)
    r = ar.Run(c, extra_tokens=4)
    out, lse = r.call().results()
    ar.check(c, (out[:c.T], lse[:c.T]))
    assert bool((out[c.T:] == 0).all()) and bool((lse[c.T:] == -math.inf).all())


@pytest.mark.parametrize("qlens", [None, [30, 5, 9]])
def test_same_bits_again(qlens):
    c = ar.make("bf16", lens=[700, 650, 1300], qlens=qlens, prefix=600, layers=1, layer=0)
    r = ar.Run(c)
    a = r.call().results()
    r.out.fill_(0)
    r.ws.fill_(255)
    b = r.call().results()
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_graph_replay_with_new_lengths():
    """A captured step replayed on other lengths and tables."""
    c = ar.make("bf16", lens=[300, 350, 0, 1000], prefix=256, layers=1, layer=0)
    d = ar.make("bf16", lens=[700, 0, 257, 999], prefix=256, layers=1, layer=0, seed=5)
    width = max(c.tables.shape[1], d.tables.shape[1])
    for x in (c, d):
        x.tables = torch.nn.functional.pad(x.tables, (0, width - x.tables.shape[1]), value=-3)
    size = max(len(c.pool), len(d.pool)) // 2
    pages = max(c.pages, d.pages)
    r = ar.Run(c if c.pages == pages else d)
    s = torch.cuda.Stream()
    def load(x):
        big = torch.zeros(2, pages * 16, x.H, x.D, dtype=torch.bfloat16)
        big[:, :x.pages * 16] = x.pool.view(torch.bfloat16).view(2, x.pages * 16, x.H, x.D)
        r.pool.copy_(big.view(torch.uint8).view(-1))
        r.tables.copy_(x.tables)
        r.prefix_pages.copy_(x.prefix_pages)
        r.lens.copy_(torch.tensor(x.lens, dtype=torch.int32))
        r.q.copy_(x.q)
    load(c)
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        r.call()
        s.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            r.call()
    for x in (d, c, d):
        load(x)
        torch.cuda.synchronize()
        g.replay()
        ar.check(x, r.results())
    assert size > 0


def test_streams_and_workspaces_of_their_own():
    cases = [ar.make("bf16", lens=[400 + i, 300], prefix=256, seed=i) for i in range(4)]
    runs = [ar.Run(c) for c in cases]
    streams = [torch.cuda.Stream() for _ in runs]
    torch.cuda.synchronize()
    for _ in range(5):
        for r, s in zip(runs, streams):
            r.call(stream=s)
    torch.cuda.synchronize()
    for c, r in zip(cases, runs):
        ar.check(c, r.results())


def _status(r, **more):
    r.call(**more)
    torch.cuda.synchronize()
    return int(r.status.item())


def test_device_refusals():
    """Bad lengths, query starts and page ids are reported; nothing outside the pool is read."""
    kvx = ar.Run(ar.make("bf16", lens=[50])).kvx
    for edit, want in [
        (lambda r: r.lens.fill_(-1), kvx.ERR_INVALID_ARG),
        (lambda r: r.lens.fill_(100000), kvx.ERR_OUT_OF_RANGE),
        (lambda r: r.tables.fill_(-1), kvx.ERR_OUT_OF_RANGE),
        (lambda r: r.tables.fill_(r.c.pages), kvx.ERR_OUT_OF_RANGE),
        (lambda r: r.prefix_pages.fill_(2 ** 31 - 1), kvx.ERR_OUT_OF_RANGE),
    ]:
        for dtype, D in (("bf16", 64), ("bf16", 128), ("fp8", 128), ("f32", 64)):
            for lens in ([300, 280], [300 + i for i in range(70)]):
                r = ar.Run(ar.make(dtype, D=D, lens=lens, prefix=250, layers=1, layer=0))
                edit(r)
                assert _status(r) == want
    for starts in ([1, 3, 5], [0, 3, 2], [0, 3, 6], [0, -1, 5], [0, 2 ** 31 - 1, 5]):
        r = ar.Run(ar.make("bf16", lens=[50, 60], qlens=[3, 2], prefix=16))
        r.q_start.copy_(torch.tensor(starts, dtype=torch.int32))
        assert _status(r) == kvx.ERR_INVALID_ARG
    # the same buffers are good for the next call
    r = ar.Run(ar.make("bf16", lens=[50, 60], prefix=16))
    good = r.tables.clone()
    r.tables.fill_(-1)
    assert _status(r) == kvx.ERR_OUT_OF_RANGE
    r.tables.copy_(good)
    ar.check(r.c, r.call().results())
