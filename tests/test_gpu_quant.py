"""kvx.store_kv and kvx.load_kv byte for byte against the definition: types, layouts, widths, strided and
paged tensors, NaN and infinities, bad and repeated indices, graphs, streams."""
import numpy as np
import pytest
import torch

from disaggregated_paged_kv_gb300 import kvx
from tests import quant_ref as qr

pytestmark = pytest.mark.gpu

TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
FILL = 0xA5


class Pool:
    """A pool of a known byte everywhere; bytes(p, slots): the head vectors of a plane's slots."""

    def __init__(self, pool="q4", kind="planes", page=16, L=2, H=2, D=64, pages=9, offset=0, slot_pad=0):
        self.pool, self.kind, self.page, self.L, self.H, self.D = pool, kind, page, L, H, D
        self.size, self.slots, self.P = qr.head_bytes(pool, D), pages * page, 2 * L
        R = H * self.size
        self.offset, self.pitch = offset, (self.P * R if kind == "slots" else R) + slot_pad
        total = offset + self.slots * self.pitch * (1 if kind == "slots" else self.P) + 64
        self.raw = torch.full((total,), FILL, dtype=torch.uint8, device="cuda")
        more = {"planes": dict(plane_stride=self.slots * self.pitch, slot_stride=self.pitch),
                "slots": dict(plane_stride=R, slot_stride=self.pitch),
                "hnd": dict(plane_stride=self.slots * R, kind=kvx.HND_PAGED, page_size=page)}[kind]
        self.layout = kvx.Layout(L, H, D, kvx.Q4 if pool == "q4" else kvx.FP8, self.slots,
                                 base=self.raw.data_ptr() + offset, **more)

    def view(self, host):
        """[planes, slots, heads, bytes] of the pool's bytes on the host (a view where it can be)."""
        R = self.H * self.size
        body = host[self.offset:]
        if self.kind == "slots":
            x = body[:self.slots * self.pitch].reshape(self.slots, self.pitch)[:, :self.P * R]
            return x.reshape(self.slots, self.P, self.H, self.size).transpose(1, 0, 2, 3)
        if self.kind == "planes":
            x = body[:self.P * self.slots * self.pitch].reshape(self.P, self.slots, self.pitch)[..., :R]
            return x.reshape(self.P, self.slots, self.H, self.size)
        x = body[:self.P * self.slots * R].reshape(self.P, -1, self.H, self.page, self.size)
        return x.transpose(0, 1, 3, 2, 4).reshape(self.P, self.slots, self.H, self.size)

    def write(self, planes):
        """Puts [planes, slots, heads, bytes] in, on the host's side; what lies between stays FILL."""
        R = self.H * self.size
        host = np.full(self.raw.numel(), FILL, np.uint8)
        body = host[self.offset:]
        if self.kind == "slots":
            x = body[:self.slots * self.pitch].reshape(self.slots, self.pitch)
            x[:, :self.P * R] = planes.transpose(1, 0, 2, 3).reshape(self.slots, -1)
        elif self.kind == "planes":
            x = body[:self.P * self.slots * self.pitch].reshape(self.P, self.slots, self.pitch)
            x[..., :R] = planes.reshape(self.P, self.slots, -1)
        else:
            x = planes.reshape(self.P, -1, self.page, self.H, self.size).transpose(0, 1, 3, 2, 4)
            body[:self.P * self.slots * R] = x.reshape(-1)
        return host


def values(g, shape, dtype, odd=True):
    """Normal numbers of several sizes, some groups constant or of zeros, some NaN and infinities."""
    x = g.standard_normal(shape, dtype=np.float32)
    x *= g.choice([1e-6, 1e-3, 1, 1, 1, 40, 3000], size=shape[:-1] + (1,)).astype(np.float32)
    if odd and x.size:
        flat = x.reshape(-1, shape[-1])
        pick = g.permutation(len(flat))
        for i, v in enumerate((0.0, -0.0, 7.25, -1e-9, 1e-30, -60000.0)):
            flat[pick[i % len(flat)]] = v
        for i, v in enumerate((np.nan, np.inf, -np.inf)):
            flat[pick[(6 + i) % len(flat)], g.integers(shape[-1])] = v
    return torch.from_numpy(x).to(TYPES[dtype])


def work(n):
    return (torch.empty(kvx.workspace_size(max(n, 1)), dtype=torch.uint8, device="cuda"),
            torch.full((1,), -1, dtype=torch.int32, device="cuda"))


def i32(x):
    return torch.from_numpy(np.asarray(x, np.int32)).cuda()


def expect_store(p, layer, k, v, slots, rows, scales):
    """The pool's bytes after the call, on a pool that held FILL."""
    planes = np.full((p.P, p.slots, p.H, p.size), FILL, np.uint8)
    for l in range(k.shape[0]):
        for kv, x in enumerate((k, v)):
            x = x[l].float().numpy()
            x = x if rows is None else x[rows]
            planes[2 * (layer + l) + kv, slots] = qr.encode(p.pool, x, scales[kv])
    return p.write(planes)


def check_store(p, dtype="bf16", n=40, layer=0, layers=1, paged=False, scales=(1.0, 1.0), seed=0, pad=0, tensor=None):
    g = np.random.default_rng(seed)
    m = n + 7 if paged else n
    k, v = (values(g, (layers, m, p.H, p.D), dtype) for _ in range(2))
    wide = torch.zeros(layers, m, 2 * p.H + 1, p.D + pad, dtype=TYPES[dtype], device="cuda")
    kd, vd = wide[:, :, :p.H, :p.D], wide[:, :, p.H:2 * p.H, :p.D]
    kd.copy_(k)
    vd.copy_(v)
    slots = g.permutation(p.slots)[:n]
    rows = g.permutation(m)[:n] if paged else None
    ws, st = work(n)
    a = (kd, vd) if layers > 1 else (kd[0], vd[0])
    sc = dict(k_scale=scales[0], v_scale=scales[1])
    kvx.store_kv(p.layout, layer, *a, i32(slots), ws, st, rows=None if rows is None else i32(rows), **sc)
    torch.cuda.synchronize()
    assert int(st.item()) == kvx.OK
    want = expect_store(p, layer, k, v, slots, rows, scales)
    got = p.raw.cpu().numpy()
    same(p, got, want)
    # and read back, into the middle of a wider tensor
    back = torch.full((layers, m, 2 * p.H + 1, p.D + pad), 3.0, dtype=TYPES[dtype], device="cuda")
    kb, vb = back[:, :, :p.H, :p.D], back[:, :, p.H:2 * p.H, :p.D]
    a = (kb, vb) if layers > 1 else (kb[0], vb[0])
    kvx.load_kv(p.layout, layer, *a, i32(slots), ws, st, rows=None if rows is None else i32(rows), **sc)
    torch.cuda.synchronize()
    assert int(st.item()) == kvx.OK
    exp = torch.full(back.shape, 3.0, dtype=TYPES[dtype])
    planes = p.view(want)
    for l in range(layers):
        for kv in range(2):
            y = torch.from_numpy(qr.decode(p.pool, planes[2 * (layer + l) + kv][slots], p.D, scales[kv])).to(TYPES[dtype])
            exp[l, torch.arange(n) if rows is None else torch.from_numpy(rows), kv * p.H:(kv + 1) * p.H, :p.D] = y
    got, exp = back.cpu(), exp
    assert bool(((got == exp) | (got.isnan() & exp.isnan())).all())


def same(p, got, want):
    """Byte for byte; what differs has to be the sign of a zero scale or low, which no value shows."""
    if np.array_equal(got, want):
        return
    a, b = p.view(got), p.view(want)
    assert p.pool == "q4", "bytes differ"
    outside = np.array_equal(p.write(a), got) and np.array_equal(p.write(b), want)
    assert outside, "bytes beside the rows differ"
    assert np.array_equal(a[..., :p.D // 2], b[..., :p.D // 2]), "codes differ"
    x, y = (np.ascontiguousarray(z[..., p.D // 2:]).view(np.uint16) for z in (a, b))
    diff = x != y
    assert bool(((x[diff] & 0x7FFF) == 0).all() and ((y[diff] & 0x7FFF) == 0).all()), "scales or lows differ"


@pytest.mark.parametrize("pool", ["q4", "fp8"])
@pytest.mark.parametrize("kind", ["planes", "slots", "hnd"])
@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
def test_types_and_layouts(pool, kind, dtype):
    check_store(Pool(pool, kind, 16, 2, 3, 128), dtype, 100, layer=1, scales=(0.25, 3.0), seed=1)


@pytest.mark.parametrize("pool,D", [("q4", d) for d in (32, 64, 96, 160, 256, 512)] +
                         [("fp8", d) for d in (1, 7, 8, 24, 64, 100, 192)])
@pytest.mark.parametrize("kind", ["planes", "hnd"])
def test_widths(pool, D, kind):
    check_store(Pool(pool, kind, 8, 1, 2, D), "bf16", 50, seed=D)


@pytest.mark.parametrize("n", [0, 1, 2, 31, 511, 512, 513, 2048, 2049, 8192, 8193, 20000])
def test_token_counts(n):
    check_store(Pool("q4", "planes", 16, 1, 1, 32, pages=1300), "bf16", n, seed=n)


@pytest.mark.parametrize("pool", ["q4", "fp8"])
@pytest.mark.parametrize("paged", [False, True])
@pytest.mark.parametrize("n", [33, 700])
def test_layers_and_rows(pool, paged, n):
    check_store(Pool(pool, "slots", 16, 5, 2, 64, pages=50), "f16", n, layer=1, layers=3, paged=paged, seed=n)


@pytest.mark.parametrize("pool", ["q4", "fp8"])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("pad", [1, 4, 8])
def test_unaligned_tensors_and_pools(pool, dtype, pad):
    """Rows of k and v at any element, planes and slots at any word (8-bit: any byte)."""
    step = 4 if pool == "q4" else 1
    check_store(Pool(pool, "planes", 4, 2, 3, 32, offset=step * 3, slot_pad=step * 5), dtype, 30, pad=pad, seed=pad)


@pytest.mark.parametrize("page", [1, 3, 24, 64])
def test_pages(page):
    check_store(Pool("q4", "hnd", page, 1, 3, 96, pages=200 // page + 1), "bf16", 150, seed=page)


def test_ties_and_ends_of_the_codes():
    """Values half way between two codes, scales that are powers of two: to even, as the definition says."""
    p = Pool("q4", "planes", 16, 1, 1, 32, pages=40)
    x = np.zeros((1, 600, 1, 32), np.float32)
    g = np.random.default_rng(5)
    for i in range(600):
        s = 2.0 ** g.integers(-20, 8)
        x[0, i, 0] = s * (g.integers(0, 31, 32) / 2)
        x[0, i, 0, :2] = 0, 15 * s
    x[0, 300:] -= 3.0
    k = torch.from_numpy(x)
    ws, st = work(600)
    slots = np.arange(600)
    kvx.store_kv(p.layout, 0, k[0].cuda(), k[0].cuda(), i32(slots), ws, st)
    torch.cuda.synchronize()
    same(p, p.raw.cpu().numpy(), expect_store(p, 0, k, k, slots, None, (1.0, 1.0)))


@pytest.mark.parametrize("n", [5, 3000, 9000])
@pytest.mark.parametrize("bad", [-1, None, 2 ** 31 - 1])
@pytest.mark.parametrize("where", ["slots", "rows"])
def test_an_index_out_of_range_writes_nothing(n, bad, where):
    p = Pool("q4", "planes", 16, 2, 2, 64, pages=700)
    g = np.random.default_rng(n)
    k = torch.zeros(n + 3, 2, 64, dtype=torch.bfloat16, device="cuda")
    slots, rows = g.permutation(p.slots)[:n], g.permutation(n + 3)[:n]
    slots[slots == n // 2] = p.slots - 1
    (slots if where == "slots" else rows)[n // 2] = (p.slots if where == "slots" else n + 3) if bad is None else bad
    ws, st = work(n)
    for call, k_ in ((kvx.store_kv, k), (kvx.load_kv, torch.full_like(k, 2.0))):
        before = k_.clone()
        call(p.layout, 0, k_, k_, i32(slots), ws, st, rows=i32(rows))
        torch.cuda.synchronize()
        assert int(st.item()) == kvx.ERR_OUT_OF_RANGE
        assert bool((p.raw == FILL).all()) and torch.equal(k_, before)


@pytest.mark.parametrize("n", [40, 3000])
def test_repeats(n):
    """A slot named twice is refused with CHECK_DUP; a load may name a slot often, but (checked) no row."""
    p = Pool("q4", "planes", 16, 1, 2, 64, pages=300)
    g = np.random.default_rng(n)
    k, v = (values(g, (1, n, 2, 64), "bf16", odd=False).cuda()[0] for _ in range(2))
    slots = g.permutation(p.slots)[:n]
    ws, st = work(n)
    kvx.store_kv(p.layout, 0, k, v, i32(slots), ws, st, flags=kvx.CHECK_DUP)
    torch.cuda.synchronize()
    assert int(st.item()) == kvx.OK
    held = p.raw.clone()
    twice = slots.copy()
    twice[n - 1] = twice[0]
    kvx.store_kv(p.layout, 0, v, k, i32(twice), ws, st, flags=kvx.CHECK_DUP)
    torch.cuda.synchronize()
    assert int(st.item()) == kvx.ERR_DUPLICATE_DST and torch.equal(p.raw, held)
    out = torch.zeros_like(k)
    kvx.load_kv(p.layout, 0, out, torch.zeros_like(k), i32(twice), ws, st, flags=kvx.CHECK_DUP)
    torch.cuda.synchronize()
    assert int(st.item()) == kvx.OK and torch.equal(out[0], out[n - 1])
    rows = np.arange(n)
    rows[1] = 0
    kvx.load_kv(p.layout, 0, out, out, i32(slots), ws, st, rows=i32(rows), flags=kvx.CHECK_DUP)
    torch.cuda.synchronize()
    assert int(st.item()) == kvx.ERR_DUPLICATE_DST


def test_a_repeated_token_may_be_stored_from_one_row():
    """Rows may repeat: two slots get the same token (a beam that splits)."""
    p = Pool("q4", "planes", 16, 1, 2, 64)
    k = values(np.random.default_rng(3), (1, 4, 2, 64), "bf16", odd=False)
    ws, st = work(6)
    slots, rows = np.array([5, 9, 70, 31, 2, 8]), np.array([1, 1, 0, 3, 3, 3])
    kvx.store_kv(p.layout, 0, k[0].cuda(), k[0].cuda(), i32(slots), ws, st, rows=i32(rows))
    torch.cuda.synchronize()
    same(p, p.raw.cpu().numpy(), expect_store(p, 0, k, k, slots, rows, (1.0, 1.0)))


def test_broadcast_rows():
    """Strides of zero: one row for all tokens and heads."""
    p = Pool("q4", "hnd", 16, 1, 3, 64)
    k = values(np.random.default_rng(4), (1, 1, 1, 64), "f32", odd=False)
    ws, st = work(20)
    slots = np.arange(20) * 3
    kd = k.cuda()[0].expand(20, 3, 64)
    kvx.store_kv(p.layout, 0, kd, kd, i32(slots), ws, st)
    torch.cuda.synchronize()
    same(p, p.raw.cpu().numpy(), expect_store(p, 0, k.expand(1, 20, 3, 64), k.expand(1, 20, 3, 64), slots, None, (1.0, 1.0)))


@pytest.mark.parametrize("n", [64, 3000])
def test_captured_and_replayed_on_another_stream(n):
    """A store and the load behind it in a graph, replayed with other rows and slots; the slots come from a
    kernel that runs just before."""
    p = Pool("q4", "planes", 16, 1, 2, 128, pages=400)
    g = np.random.default_rng(n)
    k, v = (values(g, (1, n, 2, 128), "bf16", odd=False).cuda()[0] for _ in range(2))
    plan = i32(g.permutation(p.slots)[:n])
    slots, out = torch.zeros_like(plan), (torch.empty_like(k), torch.empty_like(v))
    ws, st = work(n)
    s = torch.cuda.Stream()

    def calls():
        slots.copy_(plan)
        kvx.store_kv(p.layout, 0, k, v, slots, ws, st)
        kvx.load_kv(p.layout, 0, *out, slots, ws, st)
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        calls()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        calls()
    for i in range(3):
        k.copy_(values(g, (n, 2, 128), "bf16", odd=False))
        plan.copy_(i32(g.permutation(p.slots)[:n]))
        p.raw.fill_(FILL)
        graph.replay()
        torch.cuda.synchronize()
        assert int(st.item()) == kvx.OK
        where = plan.cpu().numpy()
        want = expect_store(p, 0, k.cpu()[None], v.cpu()[None], where, None, (1.0, 1.0))
        same(p, p.raw.cpu().numpy(), want)
        y = torch.from_numpy(qr.decode_q4(p.view(want)[0][where], 128, 1.0)).bfloat16()
        assert torch.equal(out[0].cpu(), y)


def test_two_calls_at_once():
    """Two streams, two pools, workspaces of their own."""
    pools = [Pool("q4", "planes", 16, 1, 8, 128, pages=400) for _ in range(2)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    n = 5000
    g = np.random.default_rng(8)
    ks = [values(g, (1, n, 8, 128), "bf16", odd=False) for _ in range(2)]
    dev = [k.cuda()[0] for k in ks]
    where = [g.permutation(6400)[:n] for _ in range(2)]
    at = [i32(w) for w in where]
    tools = [work(n) for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(3):
        for i in range(2):
            kvx.store_kv(pools[i].layout, 0, dev[i], dev[i], at[i], *tools[i], stream=streams[i])
    torch.cuda.synchronize()
    for i in range(2):
        same(pools[i], pools[i].raw.cpu().numpy(), expect_store(pools[i], 0, ks[i], ks[i], where[i], None, (1.0, 1.0)))


def test_planes_past_4_gib():
    """Byte offsets of a slot beyond 2^32."""
    slots = 60_000_000
    raw = torch.zeros(2 * slots * 80 + 64, dtype=torch.uint8, device="cuda")
    layout = kvx.Layout(1, 1, 128, kvx.Q4, slots, base=raw, plane_stride=slots * 80)
    k = values(np.random.default_rng(9), (1, 3, 1, 128), "bf16", odd=False)
    where = np.array([slots - 1, 0, 55_555_555])
    ws, st = work(3)
    out = torch.zeros(3, 1, 128, dtype=torch.bfloat16, device="cuda")
    kvx.store_kv(layout, 0, k[0].cuda(), k[0].cuda(), i32(where), ws, st)
    kvx.load_kv(layout, 0, out, torch.zeros_like(out), i32(where), ws, st)
    torch.cuda.synchronize()
    want = qr.encode_q4(k[0].float().numpy(), 1.0)
    for i, s in enumerate(where):
        for plane in range(2):
            a = (plane * slots + int(s)) * 80
            assert np.array_equal(raw[a:a + 80].cpu().numpy(), want[i, 0])
    assert torch.equal(out.cpu(), torch.from_numpy(qr.decode_q4(want, 128, 1.0)).bfloat16())


@pytest.mark.parametrize("kind", ["planes", "slots", "hnd"])
def test_4_bit_rows_move_as_bytes(kind):
    """Gather, scatter, transfer and a head range of a 4-bit pool: the bytes of its head vectors."""
    src, dst = Pool("q4", kind, 16, 2, 4, 128, pages=20), Pool("q4", "planes", 16, 2, 4, 128, pages=20)
    g = np.random.default_rng(11)
    body = g.integers(0, 256, (src.P, src.slots, 4, 80), dtype=np.uint8)
    src.raw.copy_(torch.from_numpy(src.write(body)))
    n = 100
    a, b = g.permutation(320)[:n], g.permutation(320)[:n]
    ws, st = work(n)
    kvx.transfer(src.layout, i32(a), dst.layout, i32(b), n, ws, st)
    torch.cuda.synchronize()
    got = dst.view(dst.raw.cpu().numpy())
    assert int(st.item()) == kvx.OK and np.array_equal(got[:, b], body[:, a])
    buf = torch.empty(4, n, 4, 80, dtype=torch.uint8, device="cuda")
    kvx.gather(src.layout, i32(a), n, buf, ws, st)
    torch.cuda.synchronize()
    assert np.array_equal(buf.cpu().numpy(), body[:, a])
    half = Pool("q4", "planes", 16, 2, 2, 128, pages=20)
    kvx.move_heads(kvx.OP_TRANSFER, src.layout, i32(a), 1, half.layout, i32(b), 0, 2, n, None, ws, st, buf_bytes=0)
    torch.cuda.synchronize()
    assert np.array_equal(half.view(half.raw.cpu().numpy())[:, b], body[:, a, 1:3])
