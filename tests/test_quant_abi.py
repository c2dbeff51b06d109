"""4-bit layouts, and what kvx_store_kv and kvx_load_kv refuse before any CUDA call (no GPU is
needed); the reference's own arithmetic."""
import ctypes
import os

import numpy as np
import pytest

from disaggregated_paged_kv_gb300 import build as kbuild
from disaggregated_paged_kv_gb300 import kvx
from tests import quant_ref as qr

A = 1 << 40  # an aligned address that is never read on the host
INV, ALIGN, WS, OVER = kvx.ERR_INVALID_ARG, kvx.ERR_ALIGNMENT, kvx.ERR_NO_WORKSPACE, kvx.ERR_OVERLAP


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(kvx.LIB_PATH):
        kbuild.build()
    return kvx.lib()


def pool(**kw):
    a = dict(num_layers=3, kv_heads=2, head_dim=64, dtype=kvx.Q4, num_slots=160, base=A, plane_stride=160 * 80)
    a.update(kw)
    return kvx.Layout(**a)


def args(**kw):
    a = dict(layer=1, n_layers=2, dtype=kvx.BF16, n=5, k=2 * A, v=3 * A, layer_stride=5 * 128, token_stride=128,
             head_stride=64, slots=A, rows=None, n_rows=0, k_scale=1.0, v_scale=1.0)
    a.update(kw)
    return kvx.CastArgs(**a)


def test_layouts(lib):
    assert pool().row_bytes == 80 and pool(head_dim=128).row_bytes == 160
    assert pool(head_dim=32).row_bytes == 40 and kvx.head_bytes(kvx.Q4, 96) == 60
    assert kvx.head_bytes(kvx.F32, 96) == 384
    for kw, code in ((dict(head_dim=48), INV), (dict(head_dim=16), INV), (dict(base=A + 2), ALIGN),
                     (dict(slot_stride=82), ALIGN), (dict(slot_stride=76), INV), (dict(dtype=6), INV)):
        with pytest.raises(kvx.KvxError) as e:
            pool(**kw)
        assert e.value.code == code, kw
    pool(slot_stride=84, base=A + 4)
    pool(kind=kvx.HND_PAGED, page_size=16)


def test_rows_of_another_form_are_not_moved(lib):
    """8-bit rows of as many elements are of another length; so are 4-bit rows of other widths."""
    q4, fp8 = pool(), pool(dtype=kvx.FP8, base=8 * A, plane_stride=160 * 128)
    size = kvx.workspace_size(16)
    assert lib.kvx_transfer(q4.handle, A, fp8.handle, A, 4, A, size, A, 0, None) == INV
    assert lib.kvx_move_heads(kvx.OP_TRANSFER, q4.handle, A, 0, fp8.handle, A, 0, 1, 4, None, 0, A, size, A, 0,
                              None) == INV


def test_struct_size(lib):
    assert ctypes.sizeof(kvx.CastArgs) == 88


CASES = [
    (dict(layer=-1), INV), (dict(layer=2), INV), (dict(n_layers=0), INV), (dict(n_layers=3), INV),
    (dict(dtype=kvx.FP8), INV), (dict(dtype=kvx.Q4), INV), (dict(dtype=0), INV), (dict(n=-1), INV),
    (dict(n=kvx.MAX_TOKENS + 1), INV), (dict(k=None), INV), (dict(v=None), INV), (dict(slots=None), INV),
    (dict(rows=A), INV), (dict(rows=A, n_rows=-3), INV), (dict(reserved=1), INV),
    (dict(layer_stride=-1), INV), (dict(token_stride=2 ** 41), INV), (dict(head_stride=-64), INV),
    (dict(token_stride=2 ** 40, rows=A, n_rows=2 ** 30), INV),
    (dict(k_scale=0.0), INV), (dict(v_scale=-1.0), INV), (dict(k_scale=float("nan")), INV),
    (dict(v_scale=float("inf")), INV), (dict(k_scale=1e-39), INV),
    (dict(k=2 * A + 1), ALIGN), (dict(v=3 * A + 1), ALIGN), (dict(slots=A + 2), ALIGN),
    (dict(rows=A + 1, n_rows=9), ALIGN), (dict(dtype=kvx.F32, k=2 * A + 2), ALIGN),
    (dict(k=A + 6 * 160 * 80 - 2), OVER), (dict(v=A - 1024), OVER),
    (dict(k=A - 40 * 128 * 2, rows=A, n_rows=41, layer_stride=0), OVER),
]


@pytest.mark.parametrize("kw,want", CASES)
def test_refusals(lib, kw, want):
    p, size = pool(), kvx.workspace_size(5)
    for call in (lib.kvx_store_kv, lib.kvx_load_kv):
        assert call(p.handle, args(**kw), A, size, A, 0, None) == want


def test_refusals_beside_the_arguments(lib):
    p, ok, size = pool(), args(), kvx.workspace_size(5)
    for call in (lib.kvx_store_kv, lib.kvx_load_kv):
        assert call(None, ok, A, size, A, 0, None) == INV
        assert call(p.handle, None, A, size, A, 0, None) == INV
        assert call(p.handle, ok, A, size, None, 0, None) == INV
        assert call(p.handle, ok, A, size, A + 2, 0, None) == INV
        assert call(p.handle, ok, A, size, A, 64, None) == INV
        assert call(p.handle, ok, None, size, A, 0, None) == WS
        assert call(p.handle, ok, A + 128, size, A, 0, None) == WS
        assert call(p.handle, ok, A, 100, A, 0, None) == WS
        for other in (pool(dtype=kvx.BF16, plane_stride=160 * 256), pool(dtype=kvx.F32, plane_stride=160 * 512),
                      pool(kv_planes=1)):
            assert call(other.handle, ok, A, size, A, 0, None) == INV


def test_attention_takes_16_bit_queries_of_a_4_bit_pool(lib):
    p = pool()
    a = kvx.AttnArgs(0, kvx.F32, 8, 5, 5, 16, 8, 0, 8, A, None, 0, 0, A, None, 2 * A, 512, 64, 3 * A, 512, 64, None,
                     0.125, 1.0, 1.0, 0)
    size = kvx.attention_workspace_size(p, 5, 5, 8, 0)
    assert size > 0
    assert lib.kvx_shared_attention(p.handle, a, A, size, A, None) == INV
    a.q_dtype = kvx.BF16
    assert lib.kvx_shared_attention(p.handle, a, A, size - 1, A, None) == WS


def test_reference_of_the_codes():
    """The bound that kvx.h states, and what the special values become.  With R the group's range and t its
    greatest magnitude, low is off by dl <= max(2^-11 t, 2^-25), scale by ds <= max(2^-11 (R + dl) / 15, 2^-25).  A
    code that is not clamped leaves scale / 2 <= (R + dl) / 30 (1 + 2^-11) + 2^-26, one clamped to 15 at most
    15 ds <= max(2^-11 (R + dl), 15 2^-25), one clamped to 0 dl; each is below
    R / 30 (1 + 2^-9) + 2^-11 t + 2^-21, 32-bit roundings (2^-20 of a code) included."""
    g = np.random.default_rng(1)
    for spread in (1e-6, 1e-3, 1.0, 300.0, 4000.0):
        x = (g.standard_normal((50, 128)) * spread + spread).astype(np.float32)
        y = qr.decode_q4(qr.encode_q4(x, 1.0), 128, 1.0)
        grp = x.reshape(50, 4, 32).astype(np.float64)
        top = np.abs(grp).max(-1)
        bound = (grp.max(-1) - grp.min(-1)) / 30 * (1 + 2.0 ** -9) + 2.0 ** -11 * top + 2.0 ** -21
        assert (np.abs(y.reshape(50, 4, 32) - grp) <= bound[..., None]).all()
    x = np.zeros((1, 96), np.float32)
    x[0, 0], x[0, 40], x[0, 70] = np.nan, np.inf, -np.inf
    y = qr.decode_q4(qr.encode_q4(x, 1.0), 96, 1.0)[0]
    assert np.isnan(y[:32]).all() and y[40] == 61440 and y[70] == -61440 and abs(y[41]) <= 2 and abs(y[71]) <= 4096
    assert (qr.decode_q4(qr.encode_q4(np.full((1, 32), 7.25, np.float32), 1.0), 32, 1.0) == 7.25).all()
    v = qr.e4m3_values()
    ok = ~np.isnan(v)
    assert (qr.encode_e4m3(v, 1.0)[ok] == np.arange(256)[ok]).all()
