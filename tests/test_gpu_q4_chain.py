"""The calls around a 4-bit pool together, as a decode instance makes them: taken over with quantisation, grown and
decoded step by step in a graph, moved as bytes into another pool, and read back."""
import numpy as np
import pytest
import torch

from disaggregated_paged_kv_gb300 import kvx
from examples import decode_4bit
from tests import attention_ref as ar
from tests import quant_ref as qr

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("heads,group,dim,page", [(2, 4, 128, 16), (8, 3, 64, 16), (3, 1, 128, 5), (1, 7, 96, 8)])
def test_hand_over_and_decode(heads, group, dim, page):
    layers, requests, prefix_pages = 2, 5, 4
    history, prompt, own, back = decode_4bit.run(requests=requests, prefix_pages=prefix_pages, page=page, layers=layers,
                                                 heads=heads, group=group, dim=dim, steps=4, seed=heads)
    prefix = prefix_pages * page
    b = qr.encode_q4(prompt.float().cpu().numpy(), 1.0)              # planes, tokens, heads, bytes
    x = torch.from_numpy(qr.decode_q4(b, dim, 1.0)).bfloat16().unflatten(0, (-1, 2)).transpose(0, 1)
    assert torch.equal(back.cpu(), x)
    # every request's own tokens in order, as the pool holds them
    ends = np.cumsum([0] + own) + prefix
    rows = [[np.concatenate([b[2 * l:2 * l + 2, :prefix], b[2 * l:2 * l + 2, ends[r]:ends[r + 1]]], 1)
             for r in range(requests)] for l in range(layers)]
    u = ar.U[torch.bfloat16]
    for qkv, out in history:
        for l in range(layers):
            y = qkv[l].float().cpu().numpy()
            new = qr.encode_q4(np.stack([y[:, group * heads:(group + 1) * heads], y[:, (group + 1) * heads:]]), 1.0)
            for r in range(requests):
                rows[l][r] = np.concatenate([rows[l][r], new[:, r:r + 1]], 1)
                code, step, low = qr.parts_q4(rows[l][r], dim)
                kv, mag = (torch.from_numpy(z).repeat_interleave(group, 2) for z in (code * step + low, code * step + np.abs(low)))
                q = torch.from_numpy(y[r, :group * heads]).double()
                s = torch.einsum("hd,nhd->hn", q, kv[0]) * dim ** -0.5
                ds = (dim + 8) * 2.0 ** -23 * dim ** -0.5 * torch.einsum("hd,nhd->hn", q.abs(), mag[0]).amax(-1)
                p = torch.softmax(s, -1)
                want = torch.einsum("hn,nhd->hd", p, kv[1])
                tol = u * want.abs() + (2.0 ** -10 + 2 * ds[:, None] + 2.0 ** -18) * torch.einsum("hn,nhd->hd", p, mag[1])
                ar._near(out[l, r].double().cpu(), want, tol, "out")


def test_a_moved_pool_answers_with_the_same_bits():
    """Attention over a 4-bit pool, and over what kvx.transfer made of it in another one with other slots."""
    g = torch.Generator(device="cuda").manual_seed(3)
    heads, group, dim, page, pages, n = 4, 2, 128, 16, 12, 150
    src, dst = (decode_4bit.Pool4(1, pages, page, heads, dim) for _ in range(2))
    k, v = (torch.randn(n, heads, dim, generator=g, device="cuda").half() for _ in range(2))
    at = torch.arange(n, device="cuda")
    tables = [torch.randperm(pages, generator=g, device="cuda").int()[None, :-(-n // page)].contiguous() for _ in range(2)]
    slots = [t[0, at // page] * page + at.int() % page for t in tables]
    q = torch.randn(1, heads * group, dim, generator=g, device="cuda").half()
    ws = torch.empty(max(kvx.workspace_size(n), kvx.attention_workspace_size(src.layout, 1, 1, heads * group, 0)),
                     dtype=torch.uint8, device="cuda")
    status = torch.full((4,), -1, dtype=torch.int32, device="cuda")
    kvx.store_kv(src.layout, 0, k, v, slots[0], ws, status[:1])
    kvx.transfer(src.layout, slots[0], dst.layout, slots[1], n, ws, status[1:2])
    out = [torch.empty_like(q) for _ in range(2)]
    lens = torch.tensor([n], dtype=torch.int32, device="cuda")
    for i, pool in enumerate((src, dst)):
        kvx.shared_attention(pool.layout, 0, q, out[i], tables[i], lens, page, ws, status[2 + i:3 + i])
    torch.cuda.synchronize()
    assert status.tolist() == [0, 0, 0, 0]
    assert torch.equal(out[0], out[1])


def test_the_example_runs():
    decode_4bit.main()
