"""A decode instance's first steps on KV that a prefill instance has finished.

Requests that share a prompt prefix were prefilled in one paged pool.  This instance gets their KV into
its own pool with libkvx's transfer, lays out its block tables and slot maps from the lengths alone, and
decodes: every step grows each request by a token (``kvx.block_tables``), stores the new K and V rows
where the slot map says (``kvx.scatter``) and answers the step's queries over the pool with the prefix
read once for the batch (``kvx.shared_attention``).  Everything stays on one stream and no step waits for
the host.

    python examples/decode_step.py
"""
import os
import sys

import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

from disaggregated_paged_kv_gb300 import kvx  # noqa: E402


class Pool:
    """One layer's K and V planes ([slots][heads][dim] each) and their layout."""

    def __init__(self, pages, page, heads, dim, fill=float("nan")):
        self.page, self.pages = page, pages
        self.kv = torch.full((2, pages * page, heads, dim), fill, dtype=torch.bfloat16, device="cuda")
        self.layout = kvx.Layout(1, heads, dim, kvx.BF16, pages * page, base=self.kv,
                                 plane_stride=pages * page * heads * dim * 2, keepalive=self.kv)


def i32(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def run(requests=6, prefix_pages=8, page=16, heads=2, group=4, dim=128, steps=4, seed=0):
    """Moves, lays out and decodes; returns (outputs of every step, what a plain computation gives)."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    prefix = prefix_pages * page
    own = [5 + 7 * i for i in range(requests)]               # prompt tokens behind the prefix
    lens = [prefix + n for n in own]
    tokens = prefix + sum(own)

    # the prefill side: every prompt token's K and V somewhere in its pool
    src = Pool(tokens // page + 8, page, heads, dim)
    src_slots = torch.randperm(src.pages * page, generator=g, device="cuda")[:tokens].int()
    kv = torch.randn(2, tokens, heads, dim, generator=g, device="cuda").bfloat16()
    src.kv[:, src_slots.long()] = kv

    # this side: pages for the prefix, once, and tables and slots for what each request has of its own
    dst = Pool(prefix_pages + requests * (max(own) + steps) // page + 2 * requests, page, heads, dim)
    free = torch.randperm(dst.pages, generator=g, device="cuda").int()
    shared, free = free[:prefix_pages].clone(), free[prefix_pages:].clone()
    width = max(lens) // page + steps + 2
    tables = torch.full((requests, width), -1, dtype=torch.int32, device="cuda")
    cursor, q_start = i32([0]), torch.empty(requests + 1, dtype=torch.int32, device="cuda")
    slots = torch.empty(max(sum(own), requests), dtype=torch.int32, device="cuda")
    now = i32(lens)
    ws = torch.empty(max(kvx.tables_workspace_size(requests), kvx.workspace_size(tokens),
                         kvx.attention_workspace_size(dst.layout, requests, requests, heads * group, prefix)),
                     dtype=torch.uint8, device="cuda")
    status = torch.zeros(4, dtype=torch.int32, device="cuda")  # a word a call
    kvx.block_tables(dst.layout, page, now, tables, free, cursor, cursor, q_start, slots, ws, status[:1],
                     prefix_pages=shared)
    at = torch.arange(prefix, device="cuda")
    dst_slots = torch.cat([shared[at // page] * page + at.int() % page, slots[:sum(own)]])
    kvx.transfer(src.layout, src_slots, dst.layout, dst_slots, tokens, ws, status[1:2])

    # decode
    buf = torch.empty(2, requests, heads, dim, dtype=torch.bfloat16, device="cuda")
    out = torch.empty(requests, heads * group, dim, dtype=torch.bfloat16, device="cuda")
    before, got, want = now.clone(), [], []
    history = [torch.cat([kv[:, :prefix], kv[:, prefix + a:prefix + a + n]], 1)
               for a, n in zip([sum(own[:i]) for i in range(requests)], own)]
    for _ in range(steps):
        # one projection's result: a token's queries, then its K and V heads
        qkv = torch.randn(requests, (group + 2) * heads, dim, generator=g, device="cuda").bfloat16()
        q, k, v = qkv.split([group * heads, heads, heads], 1)
        now.add_(1)
        kvx.block_tables(dst.layout, page, now, tables, free, cursor, cursor, q_start, slots, ws, status[:1],
                         old_lens=before)
        before.copy_(now)
        buf[0], buf[1] = k, v
        kvx.scatter(dst.layout, slots, requests, buf, ws, status[2:3])
        kvx.shared_attention(dst.layout, 0, q, out, tables, now, page, ws, status[3:],
                             prefix_pages=shared, prefix_len=prefix)
        got.append(out.clone())
        history = [torch.cat([x, torch.stack([k[b], v[b]])[:, None]], 1) for b, x in enumerate(history)]
        want.append(torch.stack([_plain(q[b], x, group) for b, x in enumerate(history)]))
    torch.cuda.synchronize()
    codes = status.tolist()
    if any(codes):
        raise kvx.KvxError(max(codes), "decode_step (device status)")
    return got, want


def _plain(q, kv, group):
    """One request's attention over its own tokens in order, in 64 bits."""
    k, v = (x.double().repeat_interleave(group, 1) for x in kv)      # tokens, heads * group, dim
    s = torch.einsum("hd,nhd->hn", q.double(), k) * q.shape[-1] ** -0.5
    return torch.einsum("hn,nhd->hd", torch.softmax(s, -1), v)


def main():
    got, want = run()
    worst = max(float((a.double() - b).abs().max()) for a, b in zip(got, want))
    print(f"{len(got)} decode steps on transferred KV: largest difference from a plain computation {worst:.2g}")
    assert worst < 0.05


if __name__ == "__main__":
    main()
