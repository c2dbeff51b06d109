"""Attention test cases and their values in 64 bits.

A case is a pool whose slots outside the requests all hold NaN, rows of tables with garbage past
their end, and queries taken as a slice of a wider tensor; :func:`reference` follows the
definition request by request over the tokens themselves (it never looks at the pool), and
:func:`check` holds a result to bounds derived from the formats.

Bounds.  With u the half spacing of the type at 1 (torch.finfo(type).eps / 2: 2^-8 for bf16's 8
significant bits, 2^-11 for f16's 11, 2^-24 for 32-bit floats' 24), a row's result differs from the exact one by at most
  out: u |out| + (u + 2 ds + 2^-18) * sum_j p_j |v_j|   (+ f16: weights below 2^-14 of the greatest
       are spaced 2^-24 apart, so 2^-24 sum_j |v_j| more)
  lse: ds + 2^-18 + 2^-22 |lse|
where ds bounds a score's error: products of 16- and 8-bit values are exact, their sum over
head_dim and the factor of scale and log2 e round in 32 bits, so
ds = (head_dim + 8) 2^-23 * scale * max_j sum_d |q_d k_jd|.  2^-18 stands for the exponential
(2 units in the last place) and sums of up to 2^5 parts of 2^12 terms in 32 bits, whose rounding
errors grow with the square root of the terms.
"""
import math

import torch

TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32,
         "fp8": torch.float8_e4m3fn}
U = {t: torch.finfo(t).eps / 2 for t in (torch.bfloat16, torch.float16, torch.float32)}


class Case:
    pass


def make(dtype="bf16", kind="planes", page=16, H=2, G=4, D=128, lens=(40,), qlens=None, prefix=0,
         layers=2, layer=1, io=None, q_gap=2, spread=1.5, seed=0, scale=None, k_scale=None,
         v_scale=None, slot_pad=0, offset=0, edit=None, room=0, starts=False):
    """lens: positions of each request, prefix included (0: a padding row); qlens: query tokens of
    each (None: single tokens).  slot_pad / offset: extra elements per slot and before plane 0.
    room: tokens that a table row has entries for, at least (garbage past the request's end).  starts: give
    the query starts although every request has a single token."""
    g = torch.Generator().manual_seed(seed)
    c = Case()
    c.dtype, c.kind, c.page, c.H, c.G, c.D, c.prefix = dtype, kind, page, H, G, D, prefix
    c.lens, c.single = list(lens), qlens is None and not starts
    c.qlens = [1] * len(lens) if qlens is None else list(qlens)
    c.layer, c.layers = layer, layers
    t = TYPES[dtype]
    c.io = io or (torch.bfloat16 if dtype == "fp8" else t)
    c.k_scale = k_scale if k_scale is not None else (0.25 if dtype == "fp8" else 1.0)
    c.v_scale = v_scale if v_scale is not None else (0.5 if dtype == "fp8" else 1.0)
    c.scale = D ** -0.5 if scale is None else scale
    B, T = len(c.lens), sum(c.qlens)
    # the tokens' K and V: [positions, H, D]; the prefix's are everyone's
    def rows(n):
        x = torch.randn(n, 2, H, D, generator=g)
        return (x * 3 if dtype == "fp8" else x).to(t)
    common = rows(prefix)
    c.kv = []
    for n in c.lens:
        mine = rows(max(0, n - prefix))
        c.kv.append(torch.cat([common.float(), mine.float()])[:n].to(t))
    c.common = common
    c.q = (torch.randn(T, G * H + q_gap, D, generator=g) * spread).to(c.io)[:, :G * H]
    if edit is not None:
        edit(c)
    # pages
    shared, full = -(-prefix // page), prefix // page
    mine = [max(0, -(-n // page) - full) for n in c.lens]
    pages = shared + sum(mine) + 2
    perm = torch.randperm(pages, generator=g).int()
    c.prefix_pages = perm[:shared].clone()
    width = max([1, -(-room // page)] + [-(-n // page) for n in c.lens]) + 2
    c.tables = torch.full((B, width + 1), 2 ** 31 - 7, dtype=torch.int32)[:, :width]
    at = shared
    for b, n in enumerate(c.lens):
        c.tables[b, :full] = -5  # not read: the prefix list has them
        for j in range(mine[b]):
            c.tables[b, full + j] = perm[at]
            at += 1
    c.pages = pages
    # the pool, NaN wherever no request has a token
    slots, P = pages * page, 2 * layers
    nan = torch.full((slots, P, H, D), math.nan).to(t)
    def put(slot, kv):
        for k in range(2):
            nan.view(torch.uint8)[slot, 2 * layer + k] = kv[k].contiguous().view(torch.uint8)
    for j in range(prefix):
        put(int(perm[j // page]) * page + j % page, common[j])
    for b, n in enumerate(c.lens):
        for j in range(prefix, n):
            put(int(c.tables[b, j // page]) * page + j % page, c.kv[b][j])
    raw = nan.view(torch.uint8)
    e = raw.shape[-1] // D
    if kind == "slots":
        wide = torch.zeros(offset * e + slots * (P * H * D + slot_pad) * e, dtype=torch.uint8)
        body = wide[offset * e:].view(slots, -1)
        body[:, :P * H * D * e] = raw.reshape(slots, -1)
        c.pool = wide
    else:
        x = raw.permute(1, 0, 2, 3)
        if kind == "hnd":
            x = x.reshape(P, pages, page, H, D * e).transpose(2, 3)
        c.pool = torch.cat([torch.zeros(offset * e, dtype=torch.uint8), x.reshape(-1)])
    c.e, c.P, c.slots, c.offset, c.slot_pad = e, P, slots, offset, slot_pad
    c.start = [0]
    for x in c.qlens:
        c.start.append(c.start[-1] + x)
    c.T = T
    return c


def layout(c, pool):
    from disaggregated_paged_kv_gb300 import kvx
    R = c.H * c.D * c.e
    t = {"bf16": kvx.BF16, "f16": kvx.F16, "f32": kvx.F32, "fp8": kvx.FP8}[c.dtype]
    base = pool.data_ptr() + c.offset * c.e
    if c.kind == "slots":
        return kvx.Layout(c.layers, c.H, c.D, t, c.slots, base=base, plane_stride=R,
                          slot_stride=c.P * R + c.slot_pad * c.e, keepalive=pool)
    more = dict(kind=kvx.HND_PAGED, page_size=c.page) if c.kind == "hnd" else {}
    return kvx.Layout(c.layers, c.H, c.D, t, c.slots, base=base, plane_stride=c.slots * R,
                      keepalive=pool, **more)


class Run:
    """The case's device buffers; call() runs the operator, results() reads them back."""

    def __init__(self, c, lse=True, extra_tokens=0):
        from disaggregated_paged_kv_gb300 import kvx
        self.c, self.kvx = c, kvx
        dev = lambda x: x.to("cuda")  # noqa: E731
        self.pool = dev(c.pool)
        self.layout = layout(c, self.pool)
        wide = torch.empty(c.T + extra_tokens, c.q.shape[1] + 2, c.D, dtype=c.io, device="cuda")
        self.q = wide[:, :c.q.shape[1]]
        self.q[:c.T] = dev(c.q)
        self.tables = dev(torch.nn.functional.pad(c.tables, (0, 3), value=-9))[:, :c.tables.shape[1]]
        self.prefix_pages = dev(c.prefix_pages)
        self.lens = torch.tensor(c.lens, dtype=torch.int32, device="cuda")
        self.q_start = torch.tensor(c.start, dtype=torch.int32, device="cuda")
        self.out = torch.full_like(wide, math.nan)[:, 1:1 + c.q.shape[1]]
        self.lse = torch.full(self.q.shape[:2], math.nan, device="cuda") if lse else None
        n = kvx.attention_workspace_size(self.layout, self.q.shape[0], len(c.lens), self.q.shape[1],
                                         c.prefix)
        self.ws = torch.full((n + 4096,), 255, dtype=torch.uint8, device="cuda")
        self.ws_bytes = n
        self.status = torch.full((1,), -1, dtype=torch.int32, device="cuda")

    def call(self, **more):
        c = self.c
        a = dict(q_start=None if c.single else self.q_start, prefix_pages=self.prefix_pages,
                 prefix_len=c.prefix, lse=self.lse, scale=c.scale, k_scale=c.k_scale,
                 v_scale=c.v_scale, ws_bytes=self.ws_bytes)
        a.update(more)
        self.kvx.shared_attention(self.layout, c.layer, self.q, self.out, self.tables, self.lens,
                                  c.page, self.ws, self.status, **a)
        return self

    def results(self):
        torch.cuda.synchronize()
        assert int(self.status.item()) == self.kvx.OK
        assert bool((self.ws[self.ws_bytes:] == 255).all()), "written past the workspace"
        return (self.out.double().cpu(), None if self.lse is None else self.lse.double().cpu())


def reference(c):
    """(out, lse, tol_out, tol_lse) in 64 bits."""
    HG = c.H * c.G
    out = torch.zeros(c.T, HG, c.D, dtype=torch.float64)
    lse = torch.full((c.T, HG), -math.inf, dtype=torch.float64)
    tol, tol_l = torch.zeros_like(out), torch.zeros_like(lse)
    u = U[c.io]
    for b, n in enumerate(c.lens):
        m = c.qlens[b]
        for i in range(m):
            see = n - m + i + 1
            if see <= 0:
                continue
            t = c.start[b] + i
            k = c.kv[b][:see, 0].double() * c.k_scale        # n, H, D
            v = c.kv[b][:see, 1].double() * c.v_scale
            q = c.q[t].double().view(c.H, c.G, c.D)
            s = torch.einsum("hgd,nhd->hgn", q, k) * c.scale
            ds = (c.D + 8) * 2.0 ** -23 * abs(c.scale) * \
                torch.einsum("hgd,nhd->hgn", q.abs(), k.abs()).amax(-1)
            p = torch.softmax(s, -1)
            o = torch.einsum("hgn,nhd->hgd", p, v)
            a = torch.einsum("hgn,nhd->hgd", p, v.abs())
            out[t] = o.reshape(HG, c.D)
            lse[t] = torch.logsumexp(s, -1).view(HG)
            e = u * o.abs() + (u + 2 * ds[..., None] + 2.0 ** -18) * a
            if c.io == torch.float16:
                e = e + 2.0 ** -24 * v.abs().sum(0)[:, None]
            tol[t] = e.reshape(HG, c.D)
            tol_l[t] = (ds + 2.0 ** -18).view(HG) + 2.0 ** -22 * lse[t].abs()
    return out, lse, tol, tol_l


def check(c, got):
    out, lse = got
    want, wlse, tol, tol_l = reference(c)
    _near(out[:c.T], want, tol, "out")
    if lse is not None:
        _near(lse[:c.T], wlse, tol_l, "lse")


def _near(got, want, tol, what):
    fine = torch.isfinite(want)
    same = torch.where(torch.isnan(want), torch.isnan(got), got == want)
    assert bool((same | fine).all()), f"{what}: infinities or NaN differ"
    bad = fine & ~((got - want).abs() <= tol)
    assert not bool(bad.any()), (
        f"{what}: {int(bad.sum())} of {bad.numel()} off, first at {bad.nonzero()[0].tolist()}, "
        f"worst {float(((got - want).abs() / tol.clamp(min=1e-30))[bad].max()):.3g} times the bound")
