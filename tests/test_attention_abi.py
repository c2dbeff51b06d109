"""kvx_block_tables and kvx_shared_attention refuse what the host can see, before any CUDA call
(no GPU is needed)."""
import ctypes
import os

import pytest

from disaggregated_paged_kv_gb300 import build as kbuild
from disaggregated_paged_kv_gb300 import kvx

A = 1 << 40  # an aligned address that is never read on the host


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(kvx.LIB_PATH):
        kbuild.build()
    return kvx.lib()


def pool(**kw):
    a = dict(num_layers=2, kv_heads=2, head_dim=64, dtype=kvx.BF16, num_slots=160, base=A,
             plane_stride=160 * 256)
    a.update(kw)
    return kvx.Layout(**a)


def hnd(page):
    return pool(kind=kvx.HND_PAGED, page_size=page)


def tables_args(**kw):
    a = dict(n_reqs=3, page_size=16, old_lens=A, new_lens=A, prefix_pages=A, n_prefix_pages=2,
             max_pages=8, tables=A, table_stride=8, free_pages=A, n_free=20, cursor=A, next_cursor=A,
             q_start=A, slots=A, positions=A, max_tokens=100)
    a.update(kw)
    return kvx.TablesArgs(**a)


def attn_args(**kw):
    # out is placed far from the pool
    a = dict(layer=1, q_dtype=kvx.BF16, q_heads=8, n_q=5, n_reqs=3, page_size=16, max_pages=8,
             prefix_len=32, table_stride=8, tables=A, prefix_pages=A, n_prefix_pages=2, seq_lens=A,
             q_start=A, q=A, q_token_stride=512, q_head_stride=64, out=2 * A, out_token_stride=512,
             out_head_stride=64, lse=A, scale=0.125, k_scale=1.0, v_scale=1.0)
    a.update(kw)
    return kvx.AttnArgs(**a)


def test_workspace_sizes(lib):
    assert kvx.tables_workspace_size(0) > 0
    assert kvx.tables_workspace_size(kvx.MAX_TABLE_REQUESTS) >= 8 * kvx.MAX_TABLE_REQUESTS
    assert kvx.tables_workspace_size(-1) == kvx.tables_workspace_size(kvx.MAX_TABLE_REQUESTS + 1) == 0
    p = pool()
    small = kvx.attention_workspace_size(p, 3, 3, 8, 0)
    assert 0 < small <= kvx.attention_workspace_size(p, 3, 3, 8, 64) <= \
        kvx.attention_workspace_size(p, 300, 30, 8, 64)
    for bad in ((-1, 3, 8, 0), (3, -1, 8, 0), (3, 3, 0, 0), (3, 3, 3, 0), (3, 3, 8, -1),
                (3, kvx.MAX_TABLE_REQUESTS + 1, 8, 0), (2 ** 30, 3, 8, 0)):
        assert kvx.attention_workspace_size(p, *bad) == 0
    assert lib.kvx_attention_workspace_size(None, 3, 3, 8, 0) == 0
    assert kvx.attention_workspace_size(pool(head_dim=257, plane_stride=1 << 30), 3, 3, 8, 0) == 0
    assert kvx.attention_workspace_size(pool(kv_planes=1), 3, 3, 8, 0) == 0


INV, ALIGN, WS = kvx.ERR_INVALID_ARG, kvx.ERR_ALIGNMENT, kvx.ERR_NO_WORKSPACE


@pytest.mark.parametrize("kw,want", [
    (dict(n_reqs=-1), INV), (dict(n_reqs=kvx.MAX_TABLE_REQUESTS + 1), INV), (dict(page_size=0), INV),
    (dict(n_prefix_pages=-1), INV), (dict(max_pages=0), INV), (dict(table_stride=7), INV),
    (dict(n_free=-1), INV), (dict(max_tokens=-1), INV), (dict(max_tokens=2 ** 31), INV),
    (dict(table_stride=2 ** 62), INV), (dict(reserved=1), INV), (dict(new_lens=None), INV),
    (dict(tables=None), INV), (dict(prefix_pages=None), INV), (dict(free_pages=None), INV),
    (dict(slots=None), INV), (dict(next_cursor=None), INV), (dict(q_start=None), INV),
    (dict(new_lens=A + 2), ALIGN), (dict(tables=A + 1), ALIGN), (dict(slots=A + 2), ALIGN),
    (dict(cursor=A + 1), ALIGN), (dict(positions=A + 2), ALIGN), (dict(old_lens=A + 2), ALIGN),
])
def test_tables_refusals(lib, kw, want):
    p = pool()
    size = kvx.tables_workspace_size(3)
    assert lib.kvx_block_tables(p.handle, tables_args(**kw), A, size, A, None) == want


def test_tables_refusals_beside_the_arguments(lib):
    p, size, ok = pool(), kvx.tables_workspace_size(3), tables_args()
    assert lib.kvx_block_tables(None, ok, A, size, A, None) == INV
    assert lib.kvx_block_tables(p.handle, None, A, size, A, None) == INV
    assert lib.kvx_block_tables(p.handle, ok, A, size, None, None) == INV
    assert lib.kvx_block_tables(p.handle, ok, A, size, A + 2, None) == ALIGN
    assert lib.kvx_block_tables(p.handle, ok, None, size, A, None) == WS
    assert lib.kvx_block_tables(p.handle, ok, A + 128, size, A, None) == WS
    assert lib.kvx_block_tables(p.handle, ok, A, size - 1, A, None) == WS
    assert lib.kvx_block_tables(hnd(8).handle, ok, A, size, A, None) == INV


@pytest.mark.parametrize("kw,want", [
    (dict(layer=-1), INV), (dict(layer=2), INV), (dict(q_dtype=kvx.F16), INV),
    (dict(q_dtype=kvx.F32), INV), (dict(q_dtype=9), INV), (dict(q_heads=0), INV), (dict(q_heads=7), INV),
    (dict(n_q=-1), INV), (dict(n_reqs=-1), INV), (dict(n_reqs=kvx.MAX_TABLE_REQUESTS + 1), INV),
    (dict(page_size=0), INV), (dict(page_size=161), INV), (dict(max_pages=0), INV),
    (dict(prefix_len=-1), INV), (dict(prefix_len=33), INV), (dict(table_stride=7), INV),
    (dict(table_stride=2 ** 60), INV), (dict(tables=None), INV), (dict(prefix_pages=None), INV),
    (dict(seq_lens=None), INV), (dict(q=None), INV), (dict(out=None), INV),
    (dict(q_start=None), INV), (dict(q_token_stride=-1), INV), (dict(out_head_stride=2 ** 50), INV),
    (dict(scale=float("nan")), INV), (dict(k_scale=float("inf")), INV), (dict(reserved=1), INV),
    (dict(reserved2=1), INV), (dict(q=A + 1), ALIGN), (dict(out=2 * A + 1), ALIGN),
    (dict(tables=A + 2), ALIGN), (dict(lse=A + 2), ALIGN), (dict(seq_lens=A + 1), ALIGN),
    (dict(q_start=A + 2), ALIGN), (dict(prefix_pages=A + 2), ALIGN),
    (dict(out=A + 3 * 160 * 256 - 2), kvx.ERR_OVERLAP), (dict(out=A + 4 * 160 * 256 - 2), kvx.ERR_OVERLAP),
])
def test_attention_refusals(lib, kw, want):
    p = pool()
    size = kvx.attention_workspace_size(p, 5, 3, 8, 33)
    assert lib.kvx_shared_attention(p.handle, attn_args(**kw), A, size, A, None) == want


def test_attention_refusals_beside_the_arguments(lib):
    p, ok = pool(), attn_args()
    size = kvx.attention_workspace_size(p, 5, 3, 8, 32)
    call = lib.kvx_shared_attention
    assert call(None, ok, A, size, A, None) == INV
    assert call(p.handle, None, A, size, A, None) == INV
    assert call(p.handle, ok, A, size, None, None) == INV
    assert call(p.handle, ok, A, size, A + 1, None) == ALIGN
    assert call(p.handle, ok, None, size, A, None) == WS
    assert call(p.handle, ok, A + 64, size, A, None) == WS
    assert call(p.handle, ok, A, size - 1, A, None) == WS
    assert call(hnd(8).handle, ok, A, size, A, None) == INV
    assert call(pool(kv_planes=1).handle, ok, A, size, A, None) == INV
    assert call(pool(dtype=kvx.FP8, plane_stride=160 * 128).handle, attn_args(q_dtype=kvx.F32), A,
                size, A, None) == INV


def test_struct_sizes(lib):
    assert ctypes.sizeof(kvx.TablesArgs) == 120
    assert ctypes.sizeof(kvx.AttnArgs) == 152
