"""kvx.block_tables against a plain loop: growth by a token and by many, new requests behind a
shared prefix, padding rows, page sizes, and refusals that leave every array as it was."""
import random

import pytest
import torch

from disaggregated_paged_kv_gb300 import kvx

pytestmark = pytest.mark.gpu


def plain(page, old, new, rows, prefix, free, cursor):
    """The definition, entry by entry; rows are changed in place."""
    q_start, slots, positions = [0], [], []
    for b, (o, n) in enumerate(zip(old, new)):
        first = o
        if o == 0 and n > 0:
            first = len(prefix) * page
            rows[b][:len(prefix)] = prefix
        for pos in range(first, n):
            if pos % page == 0:
                rows[b][pos // page] = free[cursor]
                cursor += 1
            slots.append(rows[b][pos // page] * page + pos % page)
            positions.append(pos)
        q_start.append(len(slots))
    return q_start, slots, positions, cursor


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


class Call:
    def __init__(self, page, old, new, prefix=0, cursor=0, width=None, spare=7, room=None, seed=0,
                 pool_kind="planes", misalign=0, free=None):
        r = random.Random(seed)
        self.page, self.old, self.new = page, old, new
        need = [-(-n // page) for n in new]
        held = [-(-o // page) for o in old]
        pages = prefix + sum(held) + cursor + sum(need) + spare
        ids = list(range(pages))
        r.shuffle(ids)
        self.prefix, ids = ids[:prefix], ids[prefix:]
        self.width = width or max(need + [prefix, 1]) + 2
        self.rows = [[-7] * self.width for _ in old]
        for b, h in enumerate(held):
            self.rows[b][:h] = ids[:h]
            ids = ids[h:]
        self.free = ids if free is None else ids[:free]
        self.cursor, self.pages = cursor, pages
        tokens = sum(max(0, n - (o or (prefix * page if n else 0))) for o, n in zip(old, new))
        room = tokens if room is None else room
        self.mem = torch.zeros(1, dtype=torch.uint8, device="cuda")
        if pool_kind == "hnd":
            self.layout = kvx.Layout(1, 1, 1, kvx.FP8, pages * page, kind=kvx.HND_PAGED, page_size=page,
                                     base=self.mem, plane_stride=pages * page)
        else:
            self.layout = kvx.Layout(1, 1, 1, kvx.FP8, pages * page, base=self.mem,
                                     plane_stride=pages * page)
        n = len(old)
        self.d_old, self.d_new = i32(old), i32(new)
        self.d_tables = i32(self.rows).view(n, self.width) if n else torch.zeros(0, self.width, dtype=torch.int32, device="cuda")
        self.d_prefix = i32(self.prefix)
        self.d_free, self.d_cursor = i32(self.free), i32([cursor])
        self.d_next, self.d_q = i32([-3]), i32([-3] * (n + 1))
        self.d_slots = i32([-3] * (room + misalign + 2))[misalign:misalign + room]
        self.d_pos = i32([-3] * (room + misalign + 2))[misalign:misalign + room]
        size = kvx.tables_workspace_size(n)
        self.ws = torch.full((size + 512,), 255, dtype=torch.uint8, device="cuda")
        self.ws_bytes = size
        self.status = i32([-1])

    def run(self, **more):
        a = dict(old_lens=self.d_old, prefix_pages=self.d_prefix, positions=self.d_pos,
                 ws_bytes=self.ws_bytes)
        a.update(more)
        kvx.block_tables(self.layout, self.page, self.d_new, self.d_tables, self.d_free,
                         self.d_cursor, self.d_next, self.d_q, self.d_slots, self.ws, self.status, **a)
        torch.cuda.synchronize()
        assert bool((self.ws[self.ws_bytes:] == 255).all())
        return int(self.status.item())

    def check(self):
        assert self.run() == kvx.OK
        q, s, p, c = plain(self.page, self.old, self.new, self.rows, self.prefix, self.free, self.cursor)
        assert self.d_q.tolist() == q
        assert self.d_tables.tolist() == self.rows
        assert self.d_slots.tolist()[:len(s)] == s and self.d_pos.tolist()[:len(p)] == p
        assert all(x == -3 for x in self.d_slots.tolist()[len(s):] + self.d_pos.tolist()[len(p):])
        assert self.d_next.item() == c


@pytest.mark.parametrize("page", [1, 2, 3, 16, 24, 64])
@pytest.mark.parametrize("n", [1, 2, 33, 300])
def test_growth(page, n):
    r = random.Random(n * 100 + page)
    old = [r.randint(1, 200) for _ in range(n)]
    Call(page, old, [o + r.choice((0, 1, 1, 1, 5, 40)) for o in old], cursor=r.randint(0, 9)).check()


@pytest.mark.parametrize("page,prefix", [(1, 0), (1, 5), (16, 0), (16, 3), (24, 2), (64, 1)])
@pytest.mark.parametrize("n", [1, 7, 130])
def test_new_requests(page, prefix, n):
    r = random.Random(n)
    new = [prefix * page + r.choice((0, 1, page - 1, page, page + 1, 300)) for _ in range(n)]
    Call(page, [0] * n, new, prefix, cursor=3).check()


def test_new_running_and_padding_rows_together():
    Call(16, [0, 100, 0, 16, 0, 1, 640], [50, 101, 0, 17, 48, 1, 900], prefix=3).check()


def test_no_requests_and_no_tokens():
    Call(16, [], []).check()
    Call(16, [5, 9], [5, 9]).check()
    Call(16, [0, 0], [0, 0], prefix=2).check()


@pytest.mark.parametrize("n", [1023, 1024, 1025, 5000])
def test_many_requests(n):
    r = random.Random(n)
    old = [r.choice((0, r.randint(1, 60))) for _ in range(n)]
    Call(16, old, [(o or 32) + r.randint(0, 20) for o in old], prefix=2, cursor=11).check()


def test_long_prompts():
    """Many chunks of tokens a request, more free pages than one CTA checks."""
    Call(1, [0, 0, 5], [70001, 3, 40000], prefix=2).check()
    Call(16, [0, 77], [300000, 123456]).check()


@pytest.mark.parametrize("misalign", [1, 2, 3])
def test_unaligned_outputs_and_spare_room(misalign):
    Call(16, [0, 30], [100, 77], misalign=misalign).check()
    Call(16, [0, 30], [100, 77], misalign=misalign, room=500).check()


def test_head_major_pool():
    Call(16, [0, 30], [100, 77], pool_kind="hnd").check()


def test_row_stride_no_old_lens_no_positions_no_cursor():
    c = Call(16, [0, 0, 0], [20, 0, 33], prefix=1)
    wide = torch.full((3, c.width + 5), -7, dtype=torch.int32, device="cuda")
    c.d_tables = wide[:, :c.width]
    assert c.run(old_lens=None, positions=None) == kvx.OK
    q, s, _, end = plain(16, c.old, c.new, c.rows, c.prefix, c.free, 0)
    assert c.d_q.tolist() == q and c.d_slots.tolist() == s and c.d_next.item() == end
    assert wide[:, :c.width].tolist() == c.rows and bool((wide[:, c.width:] == -7).all())
    assert bool((c.d_pos == -3).all())


def test_steps_chain_through_the_cursor_in_a_graph():
    """A captured decode step replayed: lengths grow on the device, the cursor is one word."""
    c = Call(4, [3, 8, 0], [4, 9, 0], spare=60, width=8)
    one = i32([1, 1, 0])
    c.d_next = c.d_cursor
    s = torch.cuda.Stream()
    old0, new0, cur0 = c.d_old.clone(), c.d_new.clone(), c.d_cursor.clone()
    torch.cuda.synchronize()

    def step():
        kvx.block_tables(c.layout, 4, c.d_new, c.d_tables, c.d_free, c.d_cursor, c.d_cursor, c.d_q,
                         c.d_slots, c.ws, c.status, old_lens=c.d_old, positions=c.d_pos)
        c.d_old.copy_(c.d_new)
        c.d_new.add_(one)
    with torch.cuda.stream(s):
        step()
        s.synchronize()
        c.d_old.copy_(old0), c.d_new.copy_(new0), c.d_cursor.copy_(cur0)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            step()
    torch.cuda.synchronize()
    rows, cur, old, new = c.rows, 0, list(c.old), list(c.new)
    for _ in range(13):
        g.replay()
        torch.cuda.synchronize()
        q, sl, p, cur = plain(4, old, new, rows, [], c.free, cur)
        assert int(c.status.item()) == kvx.OK
        assert c.d_slots.tolist() == sl and c.d_pos.tolist() == p and c.d_cursor.item() == cur
        old, new = list(new), [a + b for a, b in zip(new, (1, 1, 0))]
    for a, b in zip(c.d_tables.tolist(), rows):
        assert a == b


def test_refusals_leave_everything():
    def refused(c, want):
        before = [x.clone() for x in (c.d_tables, c.d_q, c.d_slots, c.d_pos, c.d_next)]
        assert c.run() == want
        for x, y in zip(before, (c.d_tables, c.d_q, c.d_slots, c.d_pos, c.d_next)):
            assert torch.equal(x, y)

    arg, rng = kvx.ERR_INVALID_ARG, kvx.ERR_OUT_OF_RANGE
    for n in (2, 1500):  # the requests before and behind are fine
        ok = [20] * n
        for b in (0, n // 2, n - 1):
            def one(old, new, want, **kw):
                o, m = list(ok), [25] * n
                o[b], m[b] = 16 if old is None else old, 40
                c = Call(16, [max(0, x) for x in o], m, width=8, **kw)
                c.d_old[b] = o[b]
                c.d_new[b] = new
                refused(c, want)
            one(30, 29, arg)
            one(-1, 10, arg)
            one(None, -5, arg)
            one(None, 2 ** 31 - 1, rng)
            one(None, 8 * 16 + 1, rng)
            one(0, 16, arg, prefix=2)
            one(0, 40, rng, room=10)
            one(0, 40, rng, free=1)
            for bad in (-1, 10 ** 6, 2 ** 31 - 1):
                c = Call(16, [20] * n, [25] * n)   # the page that is filled further
                c.d_tables[b, 1] = bad
                refused(c, rng)
                c = Call(16, [16] * n, [25] * n)   # a page handed out
                c.d_free[b] = bad
                refused(c, rng)
    c = Call(16, [0, 0], [40, 50], prefix=2)
    c.d_prefix[1] = -1
    refused(c, rng)
    for cur, want in ((-1, arg), (10 ** 6, rng)):
        c = Call(16, [0, 0], [40, 50])
        c.d_cursor.fill_(cur)
        refused(c, want)
    # ids that are not used may be anything
    c = Call(16, [20, 20], [25, 25])
    c.d_free.fill_(-1)
    c.d_tables[:, 0] = -1
    assert c.run() == kvx.OK
