"""A decode instance whose pool holds 4-bit values, from the hand-over to its steps.

A prefill instance has left requests that share a prompt prefix in a paged pool of bf16 rows.  This instance lays out
its block tables from the lengths alone, takes the tokens of all layers over in one call that quantises them on the
way (``kvx.store_kv`` with the source's slots as rows), and decodes: every step grows each request by a token
(``kvx.block_tables``), quantises the new K and V rows of each layer where the slot map says, and answers the
layer's queries over the 4-bit pool, the prefix read once for the batch (``kvx.shared_attention``).  The steps are
captured into a CUDA graph once and replayed.  At the end the tokens that the requests have are read back
(``kvx.load_kv``).

    python examples/decode_4bit.py
"""
import os
import sys

import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

from disaggregated_paged_kv_gb300 import kvx  # noqa: E402


def i32(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


class Pool4:
    """[planes][slots][heads][bytes of a head] and its layout."""

    def __init__(self, layers, pages, page, heads, dim):
        size, slots = kvx.head_bytes(kvx.Q4, dim), pages * page
        self.page, self.pages = page, pages
        self.bytes = torch.full((2 * layers, slots, heads, size), 255, dtype=torch.uint8, device="cuda")
        self.layout = kvx.Layout(layers, heads, dim, kvx.Q4, slots, base=self.bytes,
                                 plane_stride=slots * heads * size, keepalive=self.bytes)


def run(requests=5, prefix_pages=4, page=16, layers=2, heads=2, group=4, dim=128, steps=4, seed=0):
    """Takes over, decodes and reads back.  Returns what a caller may check: for every step and layer the queries,
    the new rows and the outputs, the prompt's rows, each request's own prompt length, and what was read back."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    prefix = prefix_pages * page
    own = [3 + 11 * i for i in range(requests)]              # prompt tokens behind the prefix
    tokens = prefix + sum(own)

    # the prefill side: every prompt token's K and V of all layers somewhere in its pool
    slots = tokens + 50
    src = torch.full((2 * layers, slots, heads, dim), float("nan"), dtype=torch.bfloat16, device="cuda")
    src_slots = torch.randperm(slots, generator=g, device="cuda")[:tokens].int()
    prompt = torch.randn(2 * layers, tokens, heads, dim, generator=g, device="cuda").bfloat16()
    src[:, src_slots.long()] = prompt

    # this side: pages for the prefix, once, and tables and slots for what each request has of its own
    dst = Pool4(layers, prefix_pages + requests * (max(own) + steps) // page + 2 * requests, page, heads, dim)
    free = torch.randperm(dst.pages, generator=g, device="cuda").int()
    shared, free = free[:prefix_pages].clone(), free[prefix_pages:].clone()
    tables = torch.full((requests, (prefix + max(own) + steps) // page + 2), -1, dtype=torch.int32, device="cuda")
    cursor, q_start = i32([0]), torch.empty(requests + 1, dtype=torch.int32, device="cuda")
    where = torch.empty(max(sum(own), requests), dtype=torch.int32, device="cuda")
    now = i32([prefix + n for n in own])
    ws = torch.empty(max(kvx.tables_workspace_size(requests), kvx.workspace_size(tokens),
                         kvx.attention_workspace_size(dst.layout, requests, requests, heads * group, prefix)),
                     dtype=torch.uint8, device="cuda")
    status = torch.zeros(4 + 2 * layers, dtype=torch.int32, device="cuda")  # a word a call
    kvx.block_tables(dst.layout, page, now, tables, free, cursor, cursor, q_start, where, ws, status[:1],
                     prefix_pages=shared)
    at = torch.arange(prefix, device="cuda")
    dst_slots = torch.cat([shared[at // page] * page + at.int() % page, where[:sum(own)]])
    kvx.store_kv(dst.layout, 0, src[0::2], src[1::2], dst_slots, ws, status[1:2], rows=src_slots)

    # a step of all layers, as a graph: one projection's result a layer, a token's queries, then its K and V heads
    before = now.clone()
    qkv = torch.zeros(layers, requests, (group + 2) * heads, dim, dtype=torch.bfloat16, device="cuda")
    out = torch.empty(layers, requests, heads * group, dim, dtype=torch.bfloat16, device="cuda")

    def step():
        now.add_(1)
        kvx.block_tables(dst.layout, page, now, tables, free, cursor, cursor, q_start, where, ws, status[:1],
                         old_lens=before)
        before.copy_(now)
        for layer in range(layers):
            q, k, v = qkv[layer].split([group * heads, heads, heads], 1)
            kvx.store_kv(dst.layout, layer, k, v, where[:requests], ws, status[4 + layer:5 + layer])
            kvx.shared_attention(dst.layout, layer, q, out[layer], tables, now, page, ws,
                                 status[4 + layers + layer:5 + layers + layer], prefix_pages=shared, prefix_len=prefix)

    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    history = []
    for _ in range(steps):
        qkv.copy_(torch.randn(qkv.shape, generator=g, device="cuda"))
        graph.replay()
        history.append((qkv.clone(), out.clone()))

    # what the requests have by now, prefix first, as bf16 rows
    back = torch.empty(2, layers, tokens, heads, dim, dtype=torch.bfloat16, device="cuda")
    kvx.load_kv(dst.layout, 0, back[0], back[1], dst_slots, ws, status[2:3])
    torch.cuda.synchronize()
    codes = status.tolist()
    if any(codes):
        raise kvx.KvxError(max(codes), "decode_4bit (device status)")
    return history, prompt, own, back


def main():
    history, prompt, own, back = run()
    x = prompt.unflatten(0, (-1, 2)).transpose(0, 1)
    off = float((back.float() - x.float()).abs().max())
    print(f"{len(history)} decode steps of {len(own)} requests over a 4-bit pool; rows read back differ by at most "
          f"{off:.2g} from the prefill's")
    assert off < 0.5


if __name__ == "__main__":
    main()
