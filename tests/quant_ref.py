"""What kvx_store_kv leaves in a pool and kvx_load_kv reads from it, in numpy, step by step as kvx.h says.

Every step of the definition is one operation of 32-bit floats (numpy rounds each of them once, to nearest
even), so pools are compared byte for byte.
"""
import numpy as np

GROUP = 32
MOST = np.float32(61440)
E4M3 = None  # all 256 values, filled at first use


def head_bytes(pool, D):
    return D // 8 * 5 if pool == "q4" else D


def encode_q4(x, scale):
    """uint8 [..., 5 D / 8] of float32 x [..., D]."""
    with np.errstate(all="ignore"):
        y = x * (np.float32(1) / np.float32(scale))
        g = y.reshape(*y.shape[:-1], y.shape[-1] // GROUP, GROUP)
        nan = np.isnan(g).any(-1)
        g = np.where(nan[..., None], np.float32(0), np.clip(g, -MOST, MOST))
        low = g.min(-1).astype(np.float16)
        base = low.astype(np.float32)
        reach = (g.max(-1) - base) * (np.float32(1) / np.float32(15))
        step = np.maximum(reach, np.float32(0)).astype(np.float16)
        s = step.astype(np.float32)
        r = np.where(s > 0, np.float32(1) / np.where(s > 0, s, np.float32(1)), np.float32(0))
        code = np.clip(np.rint((g - base[..., None]) * r[..., None]), 0, 15).astype(np.uint8)
    code[nan] = 0
    low_bits, step_bits = low.view(np.uint16).copy(), (step + np.float16(0)).view(np.uint16).copy()
    low_bits[nan], step_bits[nan] = 0x7FFF, 0
    code = code.reshape(*x.shape[:-1], x.shape[-1] // 2, 2)
    pairs = np.stack([step_bits, low_bits], -1).reshape(*x.shape[:-1], x.shape[-1] // 16)
    return np.concatenate([code[..., 0] | code[..., 1] << 4, np.ascontiguousarray(pairs).view(np.uint8)], -1)


def parts_q4(b, D):
    """(codes, scales, lows) as float64 [..., D] of the bytes of 4-bit head vectors."""
    code = np.stack([b[..., :D // 2] & 15, b[..., :D // 2] >> 4], -1).reshape(*b.shape[:-1], D)
    pairs = np.ascontiguousarray(b[..., D // 2:]).view(np.float16).astype(np.float64)
    pairs = np.repeat(pairs.reshape(*b.shape[:-1], D // GROUP, 2), GROUP, axis=-2)
    return code.astype(np.float64), pairs[..., 0], pairs[..., 1]


def decode_q4(b, D, scale):
    """float32 [..., D]: a fused multiply-add (the product is exact) and the plane's scale."""
    code, step, low = parts_q4(b, D)
    with np.errstate(all="ignore"):
        return (code * step + low).astype(np.float32) * np.float32(scale)


def e4m3_values():
    global E4M3
    if E4M3 is None:
        v = np.empty(256, np.float32)
        for i in range(256):
            e, m = i >> 3 & 15, i & 7
            x = m * 2.0 ** -9 if e == 0 else (8 + m) * 2.0 ** (e - 10)
            v[i] = np.nan if (i & 127) == 127 else -x if i & 128 else x
        E4M3 = v
    return E4M3


def encode_e4m3(x, scale):
    """The nearest E4M3 number by search among all of them, ties to the even mantissa."""
    v = e4m3_values()[:127].astype(np.float64)
    with np.errstate(all="ignore"):
        y = (x * (np.float32(1) / np.float32(scale))).astype(np.float64)
    a = np.clip(np.nan_to_num(np.abs(y), nan=0.0, posinf=448.0), 0, 448)
    hi = np.clip(np.searchsorted(v, a), 0, 126)
    lo = np.maximum(hi - 1, 0)
    up, down = v[hi] - a, a - v[lo]
    pick = np.where(up < down, hi, np.where(up > down, lo, np.where(hi % 2 == 0, hi, lo)))
    out = (pick | np.where(np.signbit(y), 128, 0)).astype(np.uint8)
    out[np.isnan(y)] = 0x7F
    return out


def encode(pool, x, scale):
    return encode_q4(x, scale) if pool == "q4" else encode_e4m3(x, scale)


def decode(pool, b, D, scale):
    if pool == "q4":
        return decode_q4(b, D, scale)
    return e4m3_values()[b] * np.float32(scale)
