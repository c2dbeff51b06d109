"""Every call that moves rows moves those of 4-bit pools as the bytes that they are."""
import ctypes

import numpy as np
import pytest
import torch

from disaggregated_paged_kv_gb300 import kvx
from tests.test_gpu_quant import FILL, Pool, i32, work

pytestmark = pytest.mark.gpu

KINDS = [("planes", "planes"), ("planes", "hnd"), ("hnd", "slots"), ("slots", "hnd"), ("hnd", "hnd")]


class Pair:
    """Two pools of L = 2 layers and a list of tokens to go from the one to the other."""

    def __init__(self, src_kind="planes", dst_kind="planes", D=128, H=4, n=150, seed=1, dst_H=None):
        g = np.random.default_rng(seed)
        self.src, self.dst = Pool("q4", src_kind, 16, 2, H, D, pages=20), Pool("q4", dst_kind, 16, 2, dst_H or H, D, pages=20)
        self.body = g.integers(0, 256, (4, 320, H, self.src.size), dtype=np.uint8)
        self.src.raw.copy_(torch.from_numpy(self.src.write(self.body)))
        self.n, self.a, self.b = n, g.permutation(320)[:n], g.permutation(320)[:n]
        self.ws, self.st = work(n)
        self.buf = torch.full((4, n, H, self.src.size), FILL, dtype=torch.uint8, device="cuda")

    def planes(self, n=None):
        """The second pool's planes when its first n tokens have come."""
        x = np.full((4, 320, self.dst.H, self.dst.size), FILL, np.uint8)
        x[:, self.b[:n]] = self.body[:, self.a[:n]]
        return x

    def check_dst(self, want=None):
        torch.cuda.synchronize()
        assert np.array_equal(self.dst.raw.cpu().numpy(), self.dst.write(self.planes() if want is None else want))

    def check_buf(self):
        torch.cuda.synchronize()
        assert np.array_equal(self.buf.cpu().numpy(), self.body[:, self.a])

    def ok(self, st=None):
        torch.cuda.synchronize()
        assert (self.st if st is None else st).tolist()[0] == kvx.OK


@pytest.mark.parametrize("src,dst", KINDS)
@pytest.mark.parametrize("D,H", [(128, 4), (64, 2), (96, 3), (32, 1)])
@pytest.mark.parametrize("n", [1, 3, 150])
def test_lists_of_slots(src, dst, D, H, n):
    p = Pair(src, dst, D, H, n)
    kvx.gather(p.src.layout, i32(p.a), n, p.buf, p.ws, p.st)
    p.check_buf()
    kvx.scatter(p.dst.layout, i32(p.b), n, p.buf, p.ws, p.st)
    p.ok()
    p.check_dst()
    for call in ("transfer", "noalloc", "planned"):
        p.dst.raw.fill_(FILL)
        if call == "transfer":
            kvx.transfer(p.src.layout, i32(p.a), p.dst.layout, i32(p.b), n, p.ws, p.st)
        elif call == "noalloc":
            kvx.transfer_noalloc(p.src.layout, i32(p.a), p.dst.layout, i32(p.b), n, p.st)
        else:
            kvx.plan(kvx.OP_TRANSFER, p.src.layout, i32(p.a), p.dst.layout, i32(p.b), n, p.ws, p.st)
            kvx.execute(kvx.OP_TRANSFER, p.src.layout, p.dst.layout, None, 0, n, None, p.ws, p.st)
        p.ok()
        p.check_dst()


@pytest.mark.parametrize("src,dst", KINDS)
@pytest.mark.parametrize("D,H", [(128, 4), (64, 2), (96, 3)])
def test_lists_of_runs(src, dst, D, H):
    p = Pair(src, dst, D, H, 90)
    runs = np.array([(200, 10, 40), (3, 100, 1), (50, 250, 49)], np.int32)
    p.a, p.b = (np.concatenate([np.arange(r[k], r[k] + r[2]) for r in runs]) for k in (0, 1))
    dev = torch.from_numpy(runs).cuda()
    ws = torch.empty(kvx.workspace_size(p.n, 3), dtype=torch.uint8, device="cuda")
    kvx.gather_runs(p.src.layout, dev, 3, p.n, p.buf, ws, p.st)
    p.ok()
    p.check_buf()
    kvx.scatter_runs(p.dst.layout, dev, 3, p.n, p.buf, ws, p.st)
    p.ok()
    p.check_dst()
    p.dst.raw.fill_(FILL)
    kvx.transfer_runs(p.src.layout, p.dst.layout, dev, 3, p.n, ws, p.st)
    p.ok()
    p.check_dst()


@pytest.mark.parametrize("D,H", [(128, 4), (64, 2)])
def test_a_batch(D, H):
    """A transfer, a gather and a scatter of the same pools in one call."""
    p = Pair("planes", "hnd", D, H, 120)
    R = H * p.src.size
    region = -(-4 * 40 * R // 16) * 16
    buf = torch.full((2 * region,), FILL, dtype=torch.uint8, device="cuda")
    buf[region:region + 4 * 40 * R] = torch.from_numpy(np.ascontiguousarray(p.body[:, p.a[80:]])).cuda().reshape(-1)
    reqs = (kvx.Request * 3)(kvx.Request(kvx.OP_TRANSFER, 40, 0, 0, 0), kvx.Request(kvx.OP_GATHER, 40, 40, 0, 0),
                             kvx.Request(kvx.OP_SCATTER, 40, 0, 80, region))
    dev = torch.frombuffer(bytearray(ctypes.string_at(reqs, 96)), dtype=torch.uint8).cuda()
    ws = torch.empty(kvx.workspace_size(120, 3), dtype=torch.uint8, device="cuda")
    st = torch.full((4,), -1, dtype=torch.int32, device="cuda")
    kvx.batch(p.src.layout, p.dst.layout, dev, 3, 120, i32(p.a), 120, i32(p.b), 120, buf, ws, st)
    torch.cuda.synchronize()
    assert st.tolist() == [kvx.OK] * 4
    want = p.planes(40)
    want[:, p.b[80:]] = p.body[:, p.a[80:]]
    p.check_dst(want)
    assert np.array_equal(buf[:4 * 40 * R].cpu().numpy(), p.body[:, p.a[40:80]].reshape(-1))


def test_lists_on_the_host():
    p = Pair("hnd", "planes")
    st = torch.full((1,), -1, dtype=torch.int32).pin_memory()
    a, b = (torch.from_numpy(x.astype(np.int32)).pin_memory() for x in (p.a, p.b))
    kvx.submit(kvx.OP_TRANSFER, p.src.layout, a, p.dst.layout, b, p.n, None, p.ws, st, buf_bytes=0)
    p.ok(st)
    p.check_dst()


@pytest.mark.parametrize("src,dst,D,H", [("planes", "planes", 128, 4), ("hnd", "slots", 128, 3), ("slots", "hnd", 256, 1)])
@pytest.mark.parametrize("max_ctas", [0, 24])
def test_layers_as_they_come(src, dst, D, H, max_ctas):
    p = Pair(src, dst, D, H)
    ready = torch.ones(2, dtype=torch.int32, device="cuda")
    st = torch.full((4,), -1, dtype=torch.int32, device="cuda")
    more = dict(layer_ready=ready, max_ctas=max_ctas)
    kvx.stream(kvx.OP_TRANSFER, p.src.layout, i32(p.a), p.dst.layout, i32(p.b), p.n, None, p.ws, st, buf_bytes=0, **more)
    p.ok(st)
    p.check_dst()
    kvx.stream(kvx.OP_GATHER, p.src.layout, i32(p.a), None, None, p.n, p.buf, p.ws, st, **more)
    p.ok(st)
    p.check_buf()
    p.dst.raw.fill_(FILL)
    kvx.stream(kvx.OP_SCATTER, None, None, p.dst.layout, i32(p.b), p.n, p.buf, p.ws, st, **more)
    p.ok(st)
    p.check_dst()


def test_streamed_rows_off_16_bytes_are_refused():
    """Head vectors of 40 and 60 bytes, whatever their number in a row."""
    for kind, H, D in (("hnd", 2, 64), ("planes", 2, 64), ("planes", 3, 64), ("slots", 4, 96)):
        p = Pair(kind, kind, D, H)
        st = torch.full((4,), -1, dtype=torch.int32, device="cuda")
        with pytest.raises(kvx.KvxError) as e:
            kvx.stream(kvx.OP_TRANSFER, p.src.layout, i32(p.a), p.dst.layout, i32(p.b), p.n, None, p.ws, st, buf_bytes=0)
        assert e.value.code == kvx.ERR_ALIGNMENT
        with pytest.raises(kvx.KvxError) as e:
            kvx.reshard([p.src.layout], i32(p.a), [p.dst.layout], i32(p.b), kvx.tp_plan(H, 1, 1), p.n, p.ws, p.st)
        assert e.value.code == kvx.ERR_ALIGNMENT


@pytest.mark.parametrize("src,dst", KINDS)
@pytest.mark.parametrize("D", [64, 128])
def test_ranges_of_heads(src, dst, D):
    p = Pair(src, dst, D, 4, dst_H=3)
    kvx.move_heads(kvx.OP_TRANSFER, p.src.layout, i32(p.a), 1, p.dst.layout, i32(p.b), 0, 2, p.n, None, p.ws, p.st, buf_bytes=0)
    p.ok()
    want = np.full((4, 320, 3, p.dst.size), FILL, np.uint8)
    want[:, p.b, :2] = p.body[:, p.a, 1:3]
    p.check_dst(want)


@pytest.mark.parametrize("kinds", KINDS)
@pytest.mark.parametrize("streamed", [False, True])
@pytest.mark.parametrize("src_tp,dst_tp", [(2, 1), (1, 2), (2, 4)])
def test_resharding(kinds, streamed, src_tp, dst_tp):
    """Eight heads of 128 over src_tp pools, to be eight heads over dst_tp pools."""
    g, n = np.random.default_rng(3), 100
    srcs = [Pool("q4", kinds[0], 16, 2, 8 // src_tp, 128, pages=20) for _ in range(src_tp)]
    dsts = [Pool("q4", kinds[1], 16, 2, 8 // dst_tp, 128, pages=20) for _ in range(dst_tp)]
    body = g.integers(0, 256, (4, 320, 8, 80), dtype=np.uint8)
    for i, p in enumerate(srcs):
        p.raw.copy_(torch.from_numpy(p.write(body[:, :, i * p.H:(i + 1) * p.H])))
    a, b = g.permutation(320)[:n], g.permutation(320)[:n]
    ws, _ = work(n)
    st = torch.full((4,), -1, dtype=torch.int32, device="cuda")
    move = kvx.stream_reshard if streamed else kvx.reshard
    move([p.layout for p in srcs], i32(a), [p.layout for p in dsts], i32(b), kvx.tp_plan(8, src_tp, dst_tp), n, ws, st)
    torch.cuda.synchronize()
    assert int(st[0]) == kvx.OK
    for i, p in enumerate(dsts):
        want = np.full((4, 320, p.H, 80), FILL, np.uint8)
        want[:, b] = body[:, a, i * p.H:(i + 1) * p.H]
        assert np.array_equal(p.raw.cpu().numpy(), p.write(want))
