"""Attention cases over 4-bit pools: tests/attention_ref.py's cases with their keys and values quantised.

Bounds, as derived there, with two differences.  An element is low + code * scale, and a kernel may sum the two
parts apart, so errors go with mag = |low| + code * scale in the place of |k| and |v|.  And whatever the
queries' type, weights and their products with a scale are rounded to f16 (2^-11 each) for the product with the
codes:
  out: u |out| + (2 * 2^-11 + 2 ds + 2^-18) * sum_j p_j mag_j,  ds with mag of the keys
  lse: ds + 2^-18 + 2^-22 |lse|
A general kernel that works in 32 bits is well within that.  Where many rows meet the same keys, values are rounded to
f16 in the place of the products above; keys' products are exact, as everywhere.
"""
import math

import numpy as np
import torch

from tests import attention_ref as ar
from tests import quant_ref as qr


def make(dtype="bf16", kind="planes", page=16, H=2, D=128, edit_bytes=None, shift=0.0, slot_pad=0, offset=0, **kw):
    """slot_pad, offset: bytes, multiples of four.  shift: what is added to all keys and values.  edit_bytes(b, kv):
    changes a token's bytes [tokens, 2, H, bytes] in place before they are put anywhere."""
    layers, layer = kw.get("layers", 2), kw.get("layer", 1)
    c = ar.make(dtype, "planes", page, H, D=D, **kw)
    c.kind, c.offset, c.slot_pad = kind, offset, slot_pad
    size = qr.head_bytes("q4", D)
    def quantise(x):
        b = qr.encode_q4(x.float().numpy() + np.float32(shift), 1.0)
        if edit_bytes is not None:
            edit_bytes(b)
        return b
    common = quantise(c.common)
    held = [np.concatenate([common, quantise(x[c.prefix:])])[:len(x)] for x in c.kv]
    c.kv, c.mag = [], []
    for b in held:
        code, step, low = qr.parts_q4(b, D)
        c.kv.append(torch.from_numpy(code * step + low))
        c.mag.append(torch.from_numpy(code * np.abs(step) + np.abs(low)))
    P, slots = 2 * layers, c.slots
    pool = np.full((slots, P, H, size), 0xFF, np.uint8)  # scales and lows of NaN wherever there is no token
    for j in range(c.prefix):
        pool[int(c.prefix_pages[j // page]) * page + j % page, 2 * layer:2 * layer + 2] = common[j]
    for b, n in enumerate(c.lens):
        for j in range(c.prefix, n):
            pool[int(c.tables[b, j // page]) * page + j % page, 2 * layer:2 * layer + 2] = held[b][j]
    R = H * size
    if kind == "slots":
        raw = np.zeros((slots, P * R + slot_pad), np.uint8)
        raw[:, :P * R] = pool.reshape(slots, -1)
        stride = dict(plane_stride=R, slot_stride=P * R + slot_pad)
    elif kind == "planes":
        raw = np.zeros((P, slots, R + slot_pad), np.uint8)
        raw[..., :R] = pool.transpose(1, 0, 2, 3).reshape(P, slots, R)
        stride = dict(plane_stride=slots * (R + slot_pad), slot_stride=R + slot_pad)
    else:
        raw = pool.transpose(1, 0, 2, 3).reshape(P, -1, page, H, size).transpose(0, 1, 3, 2, 4)
        stride = dict(plane_stride=slots * R, kind=1, page_size=page)
    c.pool = torch.from_numpy(np.concatenate([np.zeros(offset, np.uint8), raw.reshape(-1)]))
    c.stride, c.k_scale, c.v_scale = stride, kw.get("k_scale") or 1.0, kw.get("v_scale") or 1.0
    return c


class Run(ar.Run):
    def __init__(self, c, **kw):
        from disaggregated_paged_kv_gb300 import kvx
        plain, ar.layout = ar.layout, lambda c, pool: kvx.Layout(
            c.layers, c.H, c.D, kvx.Q4, c.slots, base=pool.data_ptr() + c.offset, keepalive=pool, **c.stride)
        try:
            super().__init__(c, **kw)
        finally:
            ar.layout = plain


def reference(c):
    HG = c.H * c.G
    out = torch.zeros(c.T, HG, c.D, dtype=torch.float64)
    lse = torch.full((c.T, HG), -math.inf, dtype=torch.float64)
    tol, tol_l = torch.zeros_like(out), torch.zeros_like(lse)
    u = ar.U[c.io]
    for b, n in enumerate(c.lens):
        m = c.qlens[b]
        for i in range(m):
            see = n - m + i + 1
            if see <= 0:
                continue
            t = c.start[b] + i
            k, v = c.kv[b][:see, 0] * c.k_scale, c.kv[b][:see, 1] * c.v_scale
            mk, mv = c.mag[b][:see, 0] * abs(c.k_scale), c.mag[b][:see, 1] * abs(c.v_scale)
            q = c.q[t].double().view(c.H, c.G, c.D)
            s = torch.einsum("hgd,nhd->hgn", q, k) * c.scale
            ds = (c.D + 8) * 2.0 ** -23 * abs(c.scale) * torch.einsum("hgd,nhd->hgn", q.abs(), mk).amax(-1)
            p = torch.softmax(s, -1)
            o = torch.einsum("hgn,nhd->hgd", p, v)
            a = torch.einsum("hgn,nhd->hgd", p, mv)
            out[t] = o.reshape(HG, c.D)
            lse[t] = torch.logsumexp(s, -1).view(HG)
            tol[t] = (u * o.abs() + (2.0 ** -10 + 2 * ds[..., None] + 2.0 ** -18) * a).reshape(HG, c.D)
            tol_l[t] = (ds + 2.0 ** -18).view(HG) + 2.0 ** -22 * lse[t].abs()
    return out, lse, tol, tol_l


def check(c, got):
    out, lse = got
    want, wlse, tol, tol_l = reference(c)
    ar._near(out[:c.T], want, tol, "out")
    if lse is not None:
        ar._near(lse[:c.T], wlse, tol_l, "lse")
