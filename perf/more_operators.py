"""What the operators of a quantised KV pool are measured on.

Three operators of a decode instance whose paged pool holds 4-bit (or 8-bit) values: rows quantised as
they are written, rows read back, and attention over a 4-bit pool.  ``listed`` names the measured cases,
``draw`` makes more of the same ranges, ``run`` is one call of an operator (the framework's where ``own``
is true, elementary torch operations otherwise) and ``exact`` the definition in 64 bits.

A 4-bit head vector of D elements is D / 2 bytes of codes (element 2 i in the low half of byte i) and, for
every 32 elements, a pair of 16-bit floats, scale and low: an element is low + code * scale.  Of 32 values
clamped to +-61440, all steps in 32 bits: low is the least, as a 16-bit float, scale the 16-bit float nearest to
(greatest - low) * (1 / 15) and at least 0, and a code (value - low) * (1 / scale), rounded to even and
clamped to 0 .. 15 (0 where scale is 0).  An 8-bit element is the E4M3 value nearest to value * (1 / the plane's scale), within +-448.
"""
import math
import random

import torch

own = False

_TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
_GROUP = 32            # elements of a 4-bit vector that share a scale
_MOST = 61440.0
_K_SCALE, _V_SCALE = 0.25, 0.5  # 8-bit pools hold the values divided by these


def _attention(name, dtype, kind, page, kv_heads, group, dim, reqs, prefix, own_lo, own_hi,
               q_lo=1, q_hi=1, empty=0, layers=2):
    return {"name": name, "op": "attention", "pool": "q4", "dtype": dtype, "kind": kind, "page": page,
            "kv_heads": kv_heads, "group": group, "dim": dim, "reqs": reqs, "prefix": prefix,
            "own_lo": own_lo, "own_hi": own_hi, "q_lo": q_lo, "q_hi": q_hi, "empty": empty,
            "layers": layers}


def _rows_case(op, name, pool, dtype, kind, page, kv_heads, dim, layers, tokens, paged=False):
    return {"name": name, "op": op, "pool": pool, "dtype": dtype, "kind": kind, "page": page,
            "kv_heads": kv_heads, "dim": dim, "layers": layers, "tokens": tokens, "paged": paged}


def listed():
    return [
        # what a decode step of three short chats on a small model (2 x 128 heads) writes of a layer, and
        # reads back as later steps see it: latency
        _rows_case("store", "write step of three", "q4", "bf16", "planes", 16, 2, 128, 1, 3),
        # the same of 96 requests into 8-bit head-major pages
        _rows_case("store", "write step 96 fp8", "fp8", "bf16", "hnd", 16, 4, 128, 1, 96),
        # a layer's rows of a chunk of prompts, head-major pages, an odd number of tokens
        _rows_case("store", "write chunk 8191", "q4", "f16", "hnd", 16, 8, 128, 1, 8191),
        # a finished prefill (2048 tokens of 36 layers, 288 MiB) from its 16-bit pool into a 4-bit one
        _rows_case("store", "hand over 2048 x 36", "q4", "bf16", "planes", 16, 8, 128, 36, 2048, True),
        # a short request's rows of 64-wide heads, for a model in 32 bits
        _rows_case("load", "read 333", "q4", "f32", "slots", 64, 8, 64, 2, 333),
        # a request of 20000 tokens of 28 layers that moves on to a 16-bit pool
        _rows_case("load", "read 20000 x 28", "q4", "bf16", "planes", 16, 2, 128, 28, 20000),
        # three short chats: a decode step's latency
        _attention("q4 chat of three", "bf16", "planes", 16, 2, 6, 128, 3, 128, 1, 61),
        # 64 requests of 1000 to 2000 tokens behind a 2048-token system prompt
        _attention("q4 decode 64", "bf16", "planes", 16, 8, 4, 128, 64, 2048, 1000, 2000),
        # head-major pages, seven queries to a head, a prefix that ends inside a page, and rows that pad
        # the batch to a captured size
        _attention("q4 decode 96", "bf16", "hnd", 16, 4, 7, 128, 96, 5003, 1, 900, empty=5),
        # one request of 131072 tokens and nothing shared: the split over a long axis
        _attention("q4 one long", "f16", "slots", 1, 8, 4, 128, 1, 0, 131072, 131072, layers=1),
        # several drafted tokens a request to verify, 64-wide heads
        _attention("q4 verify 32", "f16", "planes", 64, 8, 8, 64, 32, 8192, 9, 700, 1, 8),
        # prompts of questions on one document: hundreds of new tokens each
        _attention("q4 prompts 8", "bf16", "planes", 16, 8, 4, 128, 8, 16384, 300, 512, 300, 512),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))))


def draw(rng):
    """One more case: steps, chunks and whole requests written and read, decode steps, verification and
    prompts, over every type and layout."""
    if rng.random() < 0.5:
        while True:
            layers = rng.choice((1, 1, 2, _log(rng, 1, 36)))
            c = _rows_case(rng.choice(("store", "store", "load")), "",
                           rng.choice(("q4", "q4", "q4", "fp8")), rng.choice(("bf16", "bf16", "f16", "f32")),
                           rng.choice(("planes", "slots", "hnd")), rng.choice((1, 8, 16, 24, 64)),
                           rng.choice((1, 2, 3, 4, 8)), rng.choice((32, 64, 96, 128, 128, 256)),
                           layers, _log(rng, 1, 30000))
            c["paged"] = c["op"] == "store" and rng.random() < 0.4
            if work(c)["bytes"] <= 6e8:
                del c["name"]
                return c
    while True:
        dtype = rng.choice(("bf16", "bf16", "f16"))
        mode = rng.choice(("decode", "decode", "decode", "verify", "prompt"))
        reqs = _log(rng, 1, 256 if mode == "decode" else 64 if mode == "verify" else 8)
        prefix = rng.choice((0, _log(rng, 1, 32768), 16 * _log(rng, 1, 2048)))
        q_hi = 1 if mode == "decode" else rng.randint(2, 8) if mode == "verify" else _log(rng, 9, 512)
        q_lo = rng.randint(1, q_hi)
        own_lo = q_hi + rng.choice((0, 0, _log(rng, 1, 1000)))
        own_hi = own_lo + _log(rng, 1, 2000 if reqs > 8 else 30000)
        c = _attention("", dtype, rng.choice(("planes", "slots", "hnd")),
                       rng.choice((1, 16, 16, 32, 64, 128)), rng.choice((1, 2, 4, 8)),
                       rng.choice((1, 2, 4, 6, 7, 8)), rng.choice((64, 128, 128)), reqs, prefix,
                       own_lo, own_hi, q_lo, q_hi, rng.choice((0, 0, 1, reqs // 8)),
                       rng.randint(1, 2))
        w = work(c)
        padded = reqs * own_hi * c["kv_heads"] * (c["dim"] * 8 + c["group"] * q_hi * 12)
        if w["flops"] <= 8e11 and w["bytes"] <= 5e8 and padded <= 2e10:
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


def _vector_bytes(case):
    """Bytes of one head of one token in the pool."""
    return case["dim"] * 5 // 8 if case["pool"] == "q4" else case["dim"]


def work(case):
    size, heads, dim = _vector_bytes(case), case["kv_heads"], case["dim"]
    io = 4 if case["dtype"] == "f32" else 2
    if case["op"] != "attention":
        vectors = 2 * case["layers"] * case["tokens"] * heads
        plain = 2 if case["op"] == "store" else 1  # what comes in, what it reads back as
        return {"bytes": vectors * (size + plain * dim * io) + 4 * case["tokens"] * (1 + case["paged"]),
                "flops": 0}
    length, q = _lengths(case)
    prefix = case["prefix"]
    seen = sum(max(0, n - x + i + 1) for n, x in zip(length, q) for i in range(x))
    rows = min(prefix, max(length)) + sum(max(0, n - prefix) for n in length)
    return {"bytes": 2 * rows * heads * size + sum(q) * heads * case["group"] * (2 * dim * io + 4),
            "flops": 4 * seen * heads * case["group"] * dim}


def _i32(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def _encode(x):
    """The 4-bit vectors ([..., 5 D / 8] bytes) of 32-bit values [..., D]."""
    g = x.clamp(-_MOST, _MOST).unflatten(-1, (-1, _GROUP))
    low = g.amin(-1).half()
    scale = ((g.amax(-1) - low.float()) * torch.tensor(1 / 15, dtype=torch.float32)).clamp_(min=0).half()
    r = torch.where(scale > 0, 1 / scale.float(), 0.0)
    code = ((g - low.float().unsqueeze(-1)) * r.unsqueeze(-1)).round_().clamp_(0, 15).to(torch.uint8)
    code = code.flatten(-2).unflatten(-1, (-1, 2))
    pairs = torch.stack([scale, low], -1).view(torch.uint8).flatten(-2)
    return torch.cat([code[..., 0] | code[..., 1] << 4, pairs], -1)


def _decode(b, dim):
    """The 32-bit values [..., D] of 4-bit vectors."""
    code = torch.stack([b[..., :dim // 2] & 15, b[..., :dim // 2] >> 4], -1).flatten(-2)
    pairs = b[..., dim // 2:].contiguous().view(torch.float16).float().unflatten(-1, (-1, 2))
    g = code.float().unflatten(-1, (-1, _GROUP)) * pairs[..., :1]
    return (g + pairs[..., 1:]).flatten(-2)


def _shape(case, pages):
    P, H, size, page = 2 * case["layers"], case["kv_heads"], _vector_bytes(case), case["page"]
    return {"planes": (P, pages * page, H, size), "slots": (pages * page, P, H, size),
            "hnd": (P, pages, H, page, size)}[case["kind"]]


def _pool(case, pages, gen):
    """A pool that holds normal values, each column around a middle of its own, in every slot."""
    pool = torch.empty(_shape(case, pages), dtype=torch.uint8, device="cuda")
    vectors = pool.view(-1, pool.shape[-1])
    middle = torch.randn(case["dim"], generator=gen, device="cuda").mul_(0.5)
    step = (1 << 26) // case["dim"]
    for a in range(0, len(vectors), step):
        part = vectors[a:a + step]
        x = torch.randn(len(part), case["dim"], generator=gen, device="cuda").add_(middle)
        part.copy_(_encode(x) if case["pool"] == "q4" else
                   (x * 3.0).to(torch.float8_e4m3fn).view(torch.uint8))
    return pool


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    order = list(range(case.get("reqs", 0)))
    random.Random(seed).shuffle(order)
    return (_prepare_attention(case, gen, order) if case["op"] == "attention"
            else _prepare_rows(case, gen))


def _prepare_rows(case, gen):
    page, n, L, H, D = (case[k] for k in ("page", "tokens", "layers", "kv_heads", "dim"))
    t = _TYPES[case["dtype"]]
    held = -(-n // page)
    pages = held + held // 2 + 3
    where = torch.randperm(pages, generator=gen, device="cuda").to(torch.int32)[:held]
    at = torch.arange(n, device="cuda", dtype=torch.int32)
    s = {"op": case["op"], "case": dict(case), "pages": pages,
         "slots": where[(at // page).long()] * page + at % page,
         "k_scale": _K_SCALE if case["pool"] == "fp8" else 1.0,
         "v_scale": _V_SCALE if case["pool"] == "fp8" else 1.0,
         "k_out": torch.empty(L, n, H, D, dtype=t, device="cuda"),
         "v_out": torch.empty(L, n, H, D, dtype=t, device="cuda")}
    if case["op"] == "load":
        s["pool"] = _pool(case, pages, gen)
        return s
    s["pool"] = torch.zeros(_shape(case, pages), dtype=torch.uint8, device="cuda")
    middle = torch.randn(D, generator=gen, device="cuda").mul_(0.5)
    if case["paged"]:  # the planes of a pool of that type, the tokens anywhere in it
        m = n + n // 2 + 5
        x = torch.empty(2 * L, m, H, D, dtype=t, device="cuda")
        for p in range(2 * L):
            x[p] = torch.randn(m, H, D, generator=gen, device="cuda").add_(middle)
        s["rows"] = torch.randperm(m, generator=gen, device="cuda")[:n].to(torch.int32)
        s["k"], s["v"] = x[0::2], x[1::2]
    else:  # as a projection leaves them: a token's keys and values are slices of its q, k and v
        x = torch.randn(L, n, 4 * H, D, generator=gen, device="cuda").add_(middle).to(t)
        s["rows"] = None
        s["k"], s["v"] = x[:, :, 2 * H:3 * H], x[:, :, 3 * H:]
    return s


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
        part = prefix % page
        rows = torch.nonzero(_i32(mine) > 0).view(-1)
        page_of, last = tables[rows, full].long(), perm[full].long()
        for p in (2 * layer, 2 * layer + 1):
            if case["kind"] == "hnd":
                pool[p, page_of, :, :part] = pool[p, last, :, :part].clone()
            else:
                plane = pool[p] if case["kind"] == "planes" else pool[:, p]
                head = torch.arange(part, device="cuda")
                plane[(page_of[:, None] * page + head).view(-1)] = \
                    plane[last * page + head].repeat(len(page_of), 1, 1)
    tokens, heads = sum(q), case["kv_heads"] * case["group"]
    # queries as a projection leaves them: a token's heads are a slice of its q, k and v
    wide = torch.randn(tokens, heads + 2 * case["kv_heads"], case["dim"], generator=gen,
                       device="cuda").mul_(1.5).to(_TYPES[case["dtype"]])
    start = [0]
    for x in q:
        start.append(start[-1] + x)
    return {"op": "attention", "case": dict(case), "layer": layer, "pool": pool, "pages": pages,
            "page": page, "prefix": prefix, "q": wide[:, :heads], "tables": tables,
            "prefix_pages": perm[:shared].clone(), "len": _i32(length), "q_start": _i32(start),
            "single": max(q) == 1, "most_q": max(q), "most_own": max(1, max(length) - prefix),
            "scale": 1.0 / math.sqrt(case["dim"]), "length": length, "starts": start,
            "out": torch.empty(tokens, heads, case["dim"], dtype=wide.dtype, device="cuda"),
            "lse": torch.empty(tokens, heads, dtype=torch.float32, device="cuda")}


def run(state):
    if state["op"] == "attention":
        return (_own_attention if own else _plain_attention)(state)
    return (_own_rows if own else _plain_rows)(state)


def _layout(s):
    from disaggregated_paged_kv_gb300 import kvx
    c, slots = s["case"], s["pages"] * s["case"]["page"]
    R, P = c["kv_heads"] * _vector_bytes(c), 2 * c["layers"]
    more = {"planes": dict(plane_stride=slots * R),
            "slots": dict(plane_stride=R, slot_stride=P * R),
            "hnd": dict(plane_stride=slots * R, kind=kvx.HND_PAGED, page_size=c["page"])}
    return kvx.Layout(c["layers"], c["kv_heads"], c["dim"], kvx.Q4 if c["pool"] == "q4" else kvx.FP8,
                      slots, base=s["pool"], **more[c["kind"]])


def _own_rows(s):
    from disaggregated_paged_kv_gb300 import kvx
    if "ws" not in s:  # what a program makes once for its pool
        s["layout"] = _layout(s)
        s["ws"] = torch.empty(kvx.workspace_size(s["case"]["tokens"]), dtype=torch.uint8, device="cuda")
        s["status"] = torch.empty(2, dtype=torch.int32, device="cuda")
    scales = dict(k_scale=s["k_scale"], v_scale=s["v_scale"])
    if s["op"] == "store":
        kvx.store_kv(s["layout"], 0, s["k"], s["v"], s["slots"], s["ws"], s["status"][:1],
                     rows=s["rows"], **scales)
    kvx.load_kv(s["layout"], 0, s["k_out"], s["v_out"], s["slots"], s["ws"], s["status"][1:], **scales)
    return {"k": s["k_out"], "v": s["v_out"]}


def _place(s, plane):
    """The pool's bytes of a plane, to be indexed with what _index gives: [n, heads, bytes]."""
    return s["pool"][:, plane] if s["case"]["kind"] == "slots" else s["pool"][plane]


def _index(s, slots):
    page = s["case"]["page"]
    return (slots // page, slice(None), slots % page) if s["case"]["kind"] == "hnd" else (slots,)


def _plain_rows(s):
    c, at = s["case"], _index(s, s["slots"].long())
    for p in range(2 * c["layers"]):
        scale, plane = (s["v_scale"], s["v_out"]) if p % 2 else (s["k_scale"], s["k_out"])
        if s["op"] == "store":
            x = s["v" if p % 2 else "k"][p // 2]
            x = (x if s["rows"] is None else x[s["rows"].long()]).float() * (1.0 / scale)
            _place(s, p)[at] = _encode(x) if c["pool"] == "q4" else \
                x.clamp(-448.0, 448.0).to(torch.float8_e4m3fn).view(torch.uint8)
        b = _place(s, p)[at]
        x = _decode(b, c["dim"]) if c["pool"] == "q4" else b.view(torch.float8_e4m3fn).float()
        plane[p // 2] = x * scale
    return {"k": s["k_out"], "v": s["v_out"]}


def _own_attention(s):
    from disaggregated_paged_kv_gb300 import kvx
    if "ws" not in s:  # what a program makes once for its pool
        s["layout"] = _layout(s)
        size = kvx.attention_workspace_size(s["layout"], s["q"].shape[0], len(s["len"]),
                                            s["q"].shape[1], s["prefix"])
        s["ws"] = torch.empty(size, dtype=torch.uint8, device="cuda")
        s["status"] = torch.empty(1, dtype=torch.int32, device="cuda")
    kvx.shared_attention(s["layout"], s["layer"], s["q"], s["out"], s["tables"], s["len"],
                         s["page"], s["ws"], s["status"],
                         q_start=None if s["single"] else s["q_start"],
                         prefix_pages=s["prefix_pages"], prefix_len=s["prefix"], lse=s["lse"],
                         scale=s["scale"])
    return {"out": s["out"], "lse": s["lse"]}


def _rows(s, plane, pages, at):
    """The 32-bit [..., heads, dim] rows of a plane at offsets `at` of pages."""
    pool, D = _place(s, plane), s["case"]["dim"]
    if s["case"]["kind"] == "hnd":
        return _decode(pool[pages, :, at], D)
    return _decode(pool[pages * s["page"] + at], D)


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
    k = _rows(s, 2 * layer, pages, (at % page).expand(B, S))
    v = _rows(s, 2 * layer + 1, pages, (at % page).expand(B, S))
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


def _values(bits, dim):
    """The values of 4-bit vectors in 64 bits, group by group."""
    out = torch.empty(*bits.shape[:-1], dim, dtype=torch.float64, device=bits.device)
    words = bits[..., dim // 2:].contiguous().view(torch.float16)
    for g in range(dim // _GROUP):
        scale, low = words[..., 2 * g].double(), words[..., 2 * g + 1].double()
        mine = bits[..., g * _GROUP // 2:(g + 1) * _GROUP // 2].to(torch.float64)
        high = torch.floor(mine / 16)
        out[..., g * _GROUP:(g + 1) * _GROUP:2] = low[..., None] + (mine - 16 * high) * scale[..., None]
        out[..., g * _GROUP + 1:(g + 1) * _GROUP:2] = low[..., None] + high * scale[..., None]
    return out


def _single(x):
    """64-bit values rounded to 32 bits, as the definition's steps are."""
    return x.float().double()


def _stored(x, dim):
    """What 64-bit values [..., dim] read back as from a 4-bit pool."""
    out = torch.empty_like(x)
    for a in range(0, dim, _GROUP):
        y = x[..., a:a + _GROUP].clamp(-_MOST, _MOST)
        low = y.min(-1, keepdim=True).values.half().double()
        reach = _single(_single(y.max(-1, keepdim=True).values - low) * _single(torch.tensor(1 / 15.0).double()))
        scale = reach.clamp(min=0).float().half().double()
        inverse = _single(1 / scale.masked_fill(scale == 0, 1.0))
        code = torch.round(_single(_single(y - low) * inverse)).clamp(0, 15)
        out[..., a:a + _GROUP] = low + code.masked_fill(scale == 0, 0.0) * scale
    return out


def exact(case, seed):
    """The definition in 64 bits: a layer's rows at a time, and request by request over the keys of its
    own table row alone."""
    s = prepare(case, seed)
    page, H, D = case["page"], case["kv_heads"], case["dim"]
    if case["op"] != "attention":
        out = {"k": [], "v": []}
        slots = s["slots"].long()
        for p in range(2 * case["layers"]):
            name = "v" if p % 2 else "k"
            scale = s[name + "_scale"]
            if case["op"] == "store":
                x = s[name][p // 2]
                x = (x if s["rows"] is None else x.index_select(0, s["rows"])).double() / scale
                got = _stored(x, D) if case["pool"] == "q4" else \
                    x.clamp(-448, 448).float().to(torch.float8_e4m3fn).double()
            else:
                x = s["pool"][:, p] if case["kind"] == "slots" else s["pool"][p]
                if case["kind"] == "hnd":
                    x = x.transpose(1, 2).flatten(0, 1)
                x = x.index_select(0, slots)
                got = _values(x, D) if case["pool"] == "q4" else x.view(torch.float8_e4m3fn).double()
            out[name].append(got * scale)
        return {k: torch.stack(x) for k, x in out.items()}
    G, T = case["group"], s["q"].shape[0]
    out = torch.zeros(T, H * G, D, dtype=torch.float64, device="cuda")
    lse = torch.full((T, H * G), -math.inf, dtype=torch.float64, device="cuda")
    planes = [s["pool"][:, p] if case["kind"] == "slots" else s["pool"][p]
              for p in (2 * s["layer"], 2 * s["layer"] + 1)]
    for r, n in enumerate(s["length"]):
        a, z = s["starts"][r], s["starts"][r + 1]
        if n == 0:
            continue
        ids = s["tables"][r, :-(-n // page)].long()
        kv = []
        for x in planes:
            if case["kind"] == "hnd":
                y = x[ids].transpose(1, 2).flatten(0, 1)[:n]
            else:
                y = x.unflatten(0, (-1, page))[ids].flatten(0, 1)[:n]
            kv.append(_values(y, D))
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
