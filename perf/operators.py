"""What the block-table and shared-prefix attention operators are measured on.

Two operators of the decode side of a disaggregated server: the tables and slot maps of a paged
KV pool, made on the GPU from request lengths, and attention over such a pool for a batch whose
requests share a prefix.  ``listed`` names the measured cases, ``draw`` makes more of the same
ranges, ``run`` is one call of an operator (the framework's where ``own`` is true, elementary
torch operations otherwise) and ``exact`` the definition in 64 bits.
"""
import math
import random

import torch

own = False

_TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32,
          "fp8": torch.float8_e4m3fn}
_BYTES = {"bf16": 2, "f16": 2, "f32": 4, "fp8": 1}
_K_SCALE, _V_SCALE = 0.25, 0.5  # 8-bit pools hold the values divided by these


def _attention(name, dtype, kind, page, kv_heads, group, dim, reqs, prefix, own_lo, own_hi,
               q_lo=1, q_hi=1, empty=0, layers=2):
    return {"name": name, "op": "attention", "dtype": dtype, "kind": kind, "page": page,
            "kv_heads": kv_heads, "group": group, "dim": dim, "reqs": reqs, "prefix": prefix,
            "own_lo": own_lo, "own_hi": own_hi, "q_lo": q_lo, "q_hi": q_hi, "empty": empty,
            "layers": layers}


def _tables(name, page, reqs, prefix_pages, old_lo, old_hi, add_lo, add_hi):
    return {"name": name, "op": "tables", "page": page, "reqs": reqs,
            "prefix_pages": prefix_pages, "old_lo": old_lo, "old_hi": old_hi, "add_lo": add_lo,
            "add_hi": add_hi}


def listed():
    return [
        # three short chats on a small model (28 layers of 2 x 128 heads): a decode step's latency
        _attention("chat of three", "bf16", "planes", 16, 2, 6, 128, 3, 128, 1, 61),
        # the batch of 64 requests of 1000 to 2000 tokens behind a 2048-token system prompt
        _attention("decode 64", "bf16", "planes", 16, 8, 4, 128, 64, 2048, 1000, 2000),
        # 8-bit head-major pages, seven queries to a head, a prefix that ends inside a page, and
        # rows that pad the batch to a captured size
        _attention("decode 96 fp8", "fp8", "hnd", 16, 4, 7, 128, 96, 5003, 1, 900, empty=5),
        # a large batch on one document of 32768 tokens
        _attention("decode 256 long", "bf16", "planes", 16, 8, 4, 128, 256, 32768, 1000, 2000,
                   layers=1),
        # one request of 131072 tokens and nothing shared: the split over a long axis
        _attention("one long", "f16", "slots", 1, 8, 4, 128, 1, 0, 131072, 131072, layers=1),
        # several drafted tokens a request to verify, 64-wide heads
        _attention("verify 32", "f16", "planes", 64, 8, 8, 64, 32, 8192, 9, 700, 1, 8),
        # prompts of questions on one document: hundreds of new tokens each
        _attention("prompts 8", "bf16", "planes", 16, 8, 4, 128, 8, 16384, 300, 512, 300, 512),
        # a 32-bit pool, as used to check a model
        _attention("decode f32", "f32", "planes", 16, 2, 4, 128, 5, 1000, 1, 300),
        # one request grows by one token
        _tables("tables of one", 16, 1, 0, 777, 777, 1, 1),
        # a decode step of 256 requests
        _tables("tables step 256", 16, 256, 0, 1000, 2000, 1, 1),
        # 64 new prompts of 1000 to 2000 tokens behind a shared prefix of 2048
        _tables("tables prompts 64", 16, 64, 128, 0, 0, 1000, 2000),
        # a whole pool laid out anew, 4 million tokens
        _tables("tables refill 1024", 16, 1024, 0, 0, 0, 100, 8000),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))))


def draw(rng):
    """One more case: prompts, decode steps and verification over every type and layout."""
    if rng.random() < 0.3:
        fresh = rng.random() < 0.5
        while True:
            reqs = _log(rng, 1, 1024)
            hi = _log(rng, 1, 8000)
            old = 0 if fresh else _log(rng, 1, 8000)
            page = rng.choice((1, 8, 16, 24, 64))
            if reqs * (hi + old) <= 4_000_000:
                break
        c = _tables("", page, reqs, rng.randint(0, 200) if fresh else 0, old and max(1, old // 2),
                    old, rng.randint(0, 1) if hi > 1 else 1, hi)
        del c["name"]
        return c
    while True:
        dtype = rng.choice(("bf16", "bf16", "bf16", "f16", "f16", "fp8", "fp8", "f32"))
        kv_heads = rng.choice((1, 2, 4, 8))
        group = rng.choice((1, 2, 4, 6, 7, 8))
        dim = rng.choice((64, 128, 128))
        mode = rng.choice(("decode", "decode", "decode", "verify", "prompt"))
        reqs = _log(rng, 1, 256 if mode == "decode" else 64 if mode == "verify" else 8)
        prefix = rng.choice((0, _log(rng, 1, 32768), 16 * _log(rng, 1, 2048)))
        q_hi = 1 if mode == "decode" else rng.randint(2, 8) if mode == "verify" else _log(rng, 9, 512)
        q_lo = rng.randint(1, q_hi)
        own_lo = q_hi + rng.choice((0, 0, _log(rng, 1, 1000)))
        own_hi = own_lo + _log(rng, 1, 2000 if reqs > 8 else 30000)
        c = _attention("", dtype, rng.choice(("planes", "slots", "hnd")),
                       rng.choice((1, 16, 16, 32, 64, 128)), kv_heads, group, dim, reqs, prefix,
                       own_lo, own_hi, q_lo, q_hi, rng.choice((0, 0, 1, reqs // 8)),
                       rng.randint(1, 2))
        w = work(c)
        padded = reqs * own_hi * kv_heads * (dim * 8 + group * q_hi * 12)
        if w["flops"] <= (2e10 if dtype == "f32" else 8e11) and w["bytes"] <= 1.5e9 and padded <= 2e10:
            del c["name"]
            return c


def _spread(n, lo, hi):
    """n lengths from lo to hi, the same for every seed."""
    return [hi] if n == 1 else [lo + round((hi - lo) * ((0.6180339887 * i) % 1.0)) for i in range(n)]


def _lengths(case):
    """(tokens in the pool, query tokens) of every request of an attention case."""
    n = case["reqs"]
    q = _spread(n, case["q_lo"], case["q_hi"])[::-1]
    length = [case["prefix"] + x for x in _spread(n, case["own_lo"], case["own_hi"])]
    for i in range(min(case["empty"], n)):  # rows that only pad the batch
        length[(i * 7 + 3) % n] = 0
    return length, q


def _grown(case):
    """(old, new) lengths of every request of a tables case."""
    n, start = case["reqs"], case["prefix_pages"] * case["page"]
    old = _spread(n, case["old_lo"], case["old_hi"])
    add = _spread(n, case["add_lo"], case["add_hi"])
    return old, [(o if o else start) + a for o, a in zip(old, add)]


def work(case):
    if case["op"] == "tables":
        page, pre = case["page"], case["prefix_pages"]
        old, new = _grown(case)
        first = [o if o else pre * page for o in old]
        tokens = sum(n - f for n, f in zip(new, first))
        taken = sum(-(-n // page) - -(-f // page) for n, f in zip(new, first))
        rows = case["reqs"]
        return {"bytes": 4 * (4 * rows + 1 + 2 * tokens + 2 * taken + pre * (old.count(0) + 1)),
                "flops": 0}
    length, q = _lengths(case)
    heads, dim, prefix = case["kv_heads"] * case["group"], case["dim"], case["prefix"]
    e, io = _BYTES[case["dtype"]], 4 if case["dtype"] == "f32" else 2
    seen = sum(max(0, n - x + i + 1) for n, x in zip(length, q) for i in range(x))
    rows = min(prefix, max(length)) + sum(max(0, n - prefix) for n in length)
    return {"bytes": 2 * rows * case["kv_heads"] * dim * e + sum(q) * heads * (2 * dim * io + 4),
            "flops": 4 * seen * heads * dim}


def _i32(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    order = list(range(case["reqs"]))
    random.Random(seed).shuffle(order)
    return (_prepare_tables if case["op"] == "tables" else _prepare_attention)(case, gen, order)


def _prepare_tables(case, gen, order):
    page, pre, n = case["page"], case["prefix_pages"], case["reqs"]
    old, new = _grown(case)
    old, new = [old[i] for i in order], [new[i] for i in order]
    first = [o if o else pre * page for o in old]
    tokens = sum(b - a for a, b in zip(first, new))
    have = [-(-f // page) for f in first]
    taken = sum(-(-b // page) - h for b, h in zip(new, have))
    held = sum(h for h, o in zip(have, old) if o)
    cursor = 5
    pages = pre + held + cursor + taken + 17
    perm = torch.randperm(pages, generator=gen, device="cuda").to(torch.int32)
    width = max(max(-(-b // page) for b in new), 1) + 3
    tables = torch.full((n, width), -1, dtype=torch.int32, device="cuda")
    if held:  # what each request holds already
        row = torch.repeat_interleave(torch.arange(n), torch.tensor(have)).cuda()
        at = torch.arange(held, device="cuda") - (torch.cumsum(_i32(have), 0) - _i32(have))[row]
        tables[row, at] = perm[pre:pre + held]
    return {"op": "tables", "page": page, "pages": pages, "tokens": tokens, "taken": taken,
            "old": _i32(old), "new": _i32(new), "prefix": perm[:pre].clone(),
            "free": perm[pre + held:].clone(), "cursor": _i32([cursor]), "tables": tables,
            "q_start": torch.empty(n + 1, dtype=torch.int32, device="cuda"),
            "slots": torch.empty(max(tokens, 1), dtype=torch.int32, device="cuda"),
            "positions": torch.empty(max(tokens, 1), dtype=torch.int32, device="cuda"),
            "next": torch.empty(1, dtype=torch.int32, device="cuda"),
            "pool": torch.empty(2, pages * page, 1, 16, dtype=torch.uint8, device="cuda")}


def _pool(case, pages, gen):
    """Two planes a layer of normal values, in the case's layout; every slot holds something."""
    P, H, D, page = 2 * case["layers"], case["kv_heads"], case["dim"], case["page"]
    shape = {"planes": (P, pages * page, H, D), "slots": (pages * page, P, H, D),
             "hnd": (P, pages, H, page, D)}[case["kind"]]
    pool = torch.empty(shape, dtype=_TYPES[case["dtype"]], device="cuda")
    flat = pool.view(-1)
    for a in range(0, flat.numel(), 1 << 28):
        part = flat[a:a + (1 << 28)]
        if case["dtype"] == "fp8":
            part.copy_(torch.randn(part.numel(), generator=gen, device="cuda").mul_(3.0))
        else:
            part.normal_(generator=gen)
    return pool


def _prepare_attention(case, gen, order):
    page, prefix, n = case["page"], case["prefix"], case["reqs"]
    length, q = _lengths(case)
    length, q = [length[i] for i in order], [q[i] for i in order]
    shared = -(-prefix // page)            # pages of the common list, the last one maybe in part
    full = prefix // page                  # those that a request's own row shares
    mine = [max(0, -(-x // page) - full) for x in length]
    pages = shared + sum(mine) + 3
    perm = torch.randperm(pages, generator=gen, device="cuda").to(torch.int32)
    width = max(max(-(-x // page) for x in length), 1) + 2
    tables = torch.full((n, width), -1, dtype=torch.int32, device="cuda")
    held = _i32([1 if x else 0 for x in length])
    tables[:, :full] = torch.where(held[:, None] > 0, perm[None, :full], tables[:, :full])
    row = torch.repeat_interleave(torch.arange(n), torch.tensor(mine)).cuda()
    at = torch.arange(sum(mine), device="cuda") - (torch.cumsum(_i32(mine), 0) - _i32(mine))[row]
    tables[row, full + at] = perm[shared:shared + sum(mine)]
    pool = _pool(case, pages, gen)
    layer = case["layers"] - 1
    if prefix % page:  # a request's copy of the page that the prefix ends in: equal in its head
        at, k = torch.arange(prefix % page, device="cuda"), [2 * layer, 2 * layer + 1]
        rows = torch.nonzero(_i32(mine) > 0).view(-1)
        page_of = tables[rows, full].long()
        last = perm[full].long()
        for p in k:
            if case["kind"] == "hnd":
                bits = pool.view(torch.uint8)
                bits[p, page_of, :, :prefix % page] = bits[p, last, :, :prefix % page].clone()
            else:
                plane = (pool[p] if case["kind"] == "planes" else pool[:, p]).view(torch.uint8)
                plane[(page_of[:, None] * page + at).view(-1)] = \
                    plane[last * page + at].repeat(len(page_of), 1, 1)
    io = torch.float32 if case["dtype"] == "f32" else \
        torch.float16 if case["dtype"] == "f16" else torch.bfloat16
    tokens, heads = sum(q), case["kv_heads"] * case["group"]
    # queries as a projection leaves them: a token's heads are a slice of its q, k and v
    wide = torch.randn(tokens, heads + 2 * case["kv_heads"], case["dim"], generator=gen,
                       device="cuda").mul_(1.5).to(io)
    start = [0]
    for x in q:
        start.append(start[-1] + x)
    return {"op": "attention", "case": dict(case), "layer": layer, "pool": pool, "pages": pages,
            "page": page, "prefix": prefix, "q": wide[:, :heads], "tables": tables,
            "prefix_pages": perm[:shared].clone(), "len": _i32(length), "q_start": _i32(start),
            "single": max(q) == 1, "most_q": max(q), "most_own": max(1, max(length) - prefix),
            "scale": 1.0 / math.sqrt(case["dim"]), "length": length, "starts": start,
            "out": torch.empty(tokens, heads, case["dim"], dtype=io, device="cuda"),
            "lse": torch.empty(tokens, heads, dtype=torch.float32, device="cuda")}


def run(state):
    if state["op"] == "tables":
        return (_own_tables if own else _plain_tables)(state)
    return (_own_attention if own else _plain_attention)(state)


def _tables_out(s):
    return {"tables": s["tables"], "q_start": s["q_start"], "slots": s["slots"][:s["tokens"]],
            "positions": s["positions"][:s["tokens"]], "next": s["next"]}


def _own_tables(s):
    from disaggregated_paged_kv_gb300 import kvx
    if "ws" not in s:  # what a program makes once for its pool
        s["layout"] = kvx.Layout(1, 1, 16, kvx.FP8, s["pages"] * s["page"], base=s["pool"],
                                 plane_stride=s["pages"] * s["page"] * 16)
        s["ws"] = torch.empty(kvx.tables_workspace_size(len(s["old"])), dtype=torch.uint8,
                              device="cuda")
        s["status"] = torch.empty(1, dtype=torch.int32, device="cuda")
    kvx.block_tables(s["layout"], s["page"], s["new"], s["tables"], s["free"], s["cursor"],
                     s["next"], s["q_start"], s["slots"], s["ws"], s["status"],
                     old_lens=s["old"], prefix_pages=s["prefix"], positions=s["positions"])
    return _tables_out(s)


def _plain_tables(s):
    page, n = s["page"], len(s["old"])
    pre = len(s["prefix"])
    new, fresh = s["new"], (s["old"] == 0) & (s["new"] > 0)
    first = torch.where(fresh, pre * page, s["old"])
    have, need = (first + page - 1) // page, (new + page - 1) // page
    take, count = need - have, new - first
    s["q_start"][0] = 0
    s["q_start"][1:] = torch.cumsum(count, 0)
    before = torch.cumsum(take, 0) - take
    rows = torch.arange(n, device="cuda")
    row = torch.repeat_interleave(rows, take, output_size=s["taken"])
    k = torch.arange(s["taken"], device="cuda")
    s["tables"][:, :pre] = torch.where(fresh[:, None], s["prefix"], s["tables"][:, :pre])
    s["tables"][row, have[row] + k - before[row]] = s["free"][s["cursor"] + k]
    row = torch.repeat_interleave(rows, count, output_size=s["tokens"])
    at = torch.arange(s["tokens"], device="cuda") - s["q_start"][row] + first[row]
    s["positions"][:s["tokens"]] = at
    s["slots"][:s["tokens"]] = s["tables"][row, at // page] * page + at % page
    s["next"].copy_(s["cursor"] + take.sum())
    return _tables_out(s)


def _own_attention(s):
    from disaggregated_paged_kv_gb300 import kvx
    if "ws" not in s:  # what a program makes once for its pool
        c, slots = s["case"], s["pages"] * s["page"]
        H, D, e = c["kv_heads"], c["dim"], _BYTES[c["dtype"]]
        R, P = H * D * e, 2 * c["layers"]
        t = {"bf16": kvx.BF16, "f16": kvx.F16, "f32": kvx.F32, "fp8": kvx.FP8}[c["dtype"]]
        more = {"planes": dict(plane_stride=slots * R),
                "slots": dict(plane_stride=R, slot_stride=P * R),
                "hnd": dict(plane_stride=slots * R, kind=kvx.HND_PAGED, page_size=s["page"])}
        s["layout"] = kvx.Layout(c["layers"], H, D, t, slots, base=s["pool"], **more[c["kind"]])
        size = kvx.attention_workspace_size(s["layout"], s["q"].shape[0], len(s["len"]),
                                            s["q"].shape[1], s["prefix"])
        s["ws"] = torch.empty(size, dtype=torch.uint8, device="cuda")
        s["status"] = torch.empty(1, dtype=torch.int32, device="cuda")
        s["more"] = dict(k_scale=_K_SCALE, v_scale=_V_SCALE) if c["dtype"] == "fp8" else {}
    kvx.shared_attention(s["layout"], s["layer"], s["q"], s["out"], s["tables"], s["len"],
                         s["page"], s["ws"], s["status"],
                         q_start=None if s["single"] else s["q_start"],
                         prefix_pages=s["prefix_pages"], prefix_len=s["prefix"], lse=s["lse"],
                         scale=s["scale"], **s["more"])
    return {"out": s["out"], "lse": s["lse"]}


def _rows(s, plane, pages, at):
    """The 32-bit [..., heads, dim] rows of a plane at slots (pages, at)."""
    kind, pool = s["case"]["kind"], s["pool"]
    if s["case"]["dtype"] == "fp8":  # taken out by their bits
        pool = pool.view(torch.uint8)
    if kind == "hnd":
        got = pool[plane][pages, :, at]
    else:
        got = (pool[plane] if kind == "planes" else pool[:, plane])[pages * s["page"] + at]
    if s["case"]["dtype"] == "fp8":
        return got.view(torch.float8_e4m3fn).float() * (_V_SCALE if plane % 2 else _K_SCALE)
    return got.float()


def _part(scores, mask, v):
    """A part's greatest score, sum and weighted values; [..., keys] and [..., keys, dim]."""
    scores = scores.masked_fill_(~mask, -math.inf)
    top = scores.amax(-1)
    e = scores.sub_(top.masked_fill(top == -math.inf, 0.0).unsqueeze(-1)).exp_()
    return top, e.sum(-1), e.flatten(-3, -2).matmul(v).unflatten(-2, e.shape[-3:-1])


def _plain_attention(s):
    page, prefix, layer = s["page"], s["prefix"], s["layer"]
    H, G, D = (s["case"][k] for k in ("kv_heads", "group", "dim"))
    T, B = s["q"].shape[0], len(s["len"])
    dev = s["q"].device
    q = s["q"].float().view(T, H, G, D) * s["scale"]
    first, count = s["q_start"][:B], s["q_start"][1:] - s["q_start"][:B]
    b = torch.repeat_interleave(torch.arange(B, device=dev), count, output_size=T)
    i = torch.arange(T, device=dev) - first[b]
    sees = (s["len"] - count)[b] + i + 1
    # the requests' own keys, padded to the longest
    Q, S = s["most_q"], s["most_own"]
    at = prefix + torch.arange(S, device=dev)
    pages = s["tables"][:, (at // page).clamp(max=s["tables"].shape[1] - 1)].clamp(min=0).long()
    there = (at < s["len"][:, None])[:, :, None, None]
    k = _rows(s, 2 * layer, pages, (at % page).expand(B, S)).masked_fill_(~there, 0.0)
    v = _rows(s, 2 * layer + 1, pages, (at % page).expand(B, S)).masked_fill_(~there, 0.0)
    pad = (first[:, None] + torch.arange(Q, device=dev)).clamp(max=T - 1)
    qp = q[pad].permute(0, 2, 1, 3, 4)                               # B, H, Q, G, D
    mask = at < ((s["len"] - count)[:, None] + torch.arange(Q, device=dev) + 1)[..., None]
    sc = qp.flatten(2, 3).matmul(k.permute(0, 2, 3, 1)).unflatten(2, (Q, G))
    m, l, o = _part(sc, mask[:, None, :, None, :], v.permute(0, 2, 1, 3))
    m, l, o = m[b, :, i], l[b, :, i], o[b, :, i]                     # T, H, G (, D)
    del sc, k, v, qp
    if prefix:
        at = torch.arange(prefix, device=dev)
        pages = s["prefix_pages"][at // page].long()
        k = _rows(s, 2 * layer, pages, at % page).permute(1, 2, 0)   # H, D, P
        v = _rows(s, 2 * layer + 1, pages, at % page).permute(1, 0, 2)
        sc = q.permute(1, 0, 2, 3).flatten(1, 2).matmul(k).unflatten(1, (T, G))
        m1, l1, o1 = _part(sc, (at < sees[:, None])[None, :, None, :], v)
        del sc
        m1, l1, o1 = (x.transpose(0, 1) for x in (m1, l1, o1))
        top = torch.maximum(m, m1)
        base = top.masked_fill(top == -math.inf, 0.0)
        w, w1 = torch.exp(m - base), torch.exp(m1 - base)
        m, l, o = top, l * w + l1 * w1, o * w.unsqueeze(-1) + o1 * w1.unsqueeze(-1)
    some = l > 0
    s["out"].copy_(torch.where(some.unsqueeze(-1), o / l.unsqueeze(-1), 0.0).view(T, H * G, D))
    s["lse"].copy_(torch.where(some, m + torch.log(l), -math.inf).view(T, H * G))
    return {"out": s["out"], "lse": s["lse"]}


def exact(case, seed):
    """Request by request in 64 bits, over the keys of its own table row alone."""
    if case["op"] == "tables":
        return None  # whole numbers
    s = prepare(case, seed)
    page, H, G, D = case["page"], case["kv_heads"], case["group"], case["dim"]
    T = s["q"].shape[0]
    out = torch.zeros(T, H * G, D, dtype=torch.float64, device="cuda")
    lse = torch.full((T, H * G), -math.inf, dtype=torch.float64, device="cuda")
    planes = []
    for p in (2 * s["layer"], 2 * s["layer"] + 1):
        x = s["pool"][:, p] if case["kind"] == "slots" else s["pool"][p]
        planes.append(x.view(torch.uint8) if case["dtype"] == "fp8" else x)
    for r, n in enumerate(s["length"]):
        a, z = s["starts"][r], s["starts"][r + 1]
        if n == 0:
            continue
        ids = s["tables"][r, :-(-n // page)].long()
        kv = []
        for x in planes:
            if case["kind"] == "hnd":
                y = x[ids].transpose(1, 2).reshape(-1, H, D)[:n]
            else:
                y = x.unflatten(0, (-1, page))[ids].reshape(-1, H, D)[:n]
            kv.append((y.view(torch.float8_e4m3fn).float() if case["dtype"] == "fp8" else y).double())
        if case["dtype"] == "fp8":
            kv[0] *= _K_SCALE
            kv[1] *= _V_SCALE
        for h in range(H):
            q = s["q"][a:z, h * G:(h + 1) * G].double()
            sc = torch.einsum("tgd,nd->tgn", q, kv[0][:, h]) * s["scale"]
            late = torch.arange(n, device="cuda")[None, :] > \
                (n - (z - a) + torch.arange(z - a, device="cuda"))[:, None]
            sc.masked_fill_(late[:, None], -math.inf)
            lse[a:z, h * G:(h + 1) * G] = torch.logsumexp(sc, -1)
            out[a:z, h * G:(h + 1) * G] = torch.einsum("tgn,nd->tgd", torch.softmax(sc, -1),
                                                       kv[1][:, h])
    return {"out": out, "lse": lse}
