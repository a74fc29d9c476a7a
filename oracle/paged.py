"""The paged KV cache in plain NumPy, from the definitions in include/spa.h: the 4-bit row format, the
rotation, and attention in binary64.  Test infrastructure; it shares no code with the library."""
from __future__ import annotations

import numpy as np


def bf16_bits(x):
    """Nearest-even bf16 bit patterns of fp32 values."""
    u = np.asarray(x, np.float32).view(np.uint32).astype(np.uint64)
    return ((u + 0x7FFF + ((u >> 16) & 1)) >> 16).astype(np.uint16)


def bf16_value(bits):
    return (np.asarray(bits, np.uint16).astype(np.uint32) << 16).view(np.float32)


def nibble_places(d):
    """(key, value) nibble index (2 * byte + high) of each of the d channels, from the format's table."""
    kp, vp = np.empty(d, np.int64), np.empty(d, np.int64)
    for c in range(d):
        g, j = divmod(c, d // 4)
        kp[c] = 2 * ((j // (d // 16)) * (d // 8) + g * (d // 32) + (j % (d // 16)) // 2) + j % 2
        vp[c] = 2 * ((j % 8) * (d // 16) + g * (d // 64) + j // 16) + (0 if j % 16 < 8 else 1)
    return kp, vp


def quantise(x):
    """fp32 rows [..., d] -> (codes 1..15 [..., d], scales [..., 4] fp32 holding bf16 values)."""
    x = np.asarray(x, np.float32)
    d = x.shape[-1]
    g = x.reshape(*x.shape[:-1], 4, d // 4)
    with np.errstate(all="ignore"):
        fin = np.isfinite(g).all(-1)
        top = np.where(fin, np.abs(np.where(np.isfinite(g), g, 0)).max(-1), 0).astype(np.float32)
        q = (top / np.float32(7)).astype(np.float32)
        s = ((q.view(np.uint32).astype(np.uint64) + 0xFFFF) & 0xFFFF0000).astype(np.uint32).view(np.float32)
        ok = (fin & (s > 0))[..., None]
        code = np.where(ok, np.rint((g / np.where(s > 0, s, 1)[..., None]).astype(np.float32)), 0) + 8
    s = np.where(fin, s, np.float32(np.nan)).astype(np.float32)
    return np.where(ok, code, 8).astype(np.uint8).reshape(x.shape), s


def pack(k, v):
    """fp32 keys and values [..., d] -> 4-bit rows [..., d + 16] uint8."""
    d = k.shape[-1]
    kp, vp = nibble_places(d)
    rows = np.zeros((*k.shape[:-1], d + 16), np.uint8)
    for i, (x, place) in enumerate(((k, kp), (v, vp))):
        code, s = quantise(x)
        nib = np.zeros(code.shape, np.uint8)
        nib[..., place] = code
        rows[..., i * d // 2:(i + 1) * d // 2] = nib[..., 0::2] | (nib[..., 1::2] << 4)
        bits = np.where(np.isnan(s), 0x7FC0, bf16_bits(np.nan_to_num(s))).astype("<u2")
        rows[..., d + 8 * i:d + 8 * i + 8] = np.ascontiguousarray(bits).view(np.uint8)
    return rows


def unpack(rows):
    """4-bit rows [..., d + 16] -> (keys, values) [..., d] in binary64, and their scales [..., 4]."""
    d = rows.shape[-1] - 16
    out, scales = [], []
    for i, place in enumerate(nibble_places(d)):
        by = rows[..., i * d // 2:(i + 1) * d // 2]
        nib = np.empty((*by.shape[:-1], d), np.uint8)
        nib[..., 0::2], nib[..., 1::2] = by & 15, by >> 4
        s = bf16_value(np.ascontiguousarray(rows[..., d + 8 * i:d + 8 * i + 8]).view("<u2")).astype(np.float64)
        out.append((nib[..., place].astype(np.float64) - 8) * np.repeat(s, d // 4, -1))
        scales.append(s)
    return out[0], out[1], scales[0], scales[1]


def rotate(x, pos, inv_freq, interleaved):
    """x [T, H, d] binary64 rotated by pos [T] * inv_freq [rot / 2]."""
    y = np.array(x, np.float64)
    half = len(inv_freq)
    a = np.asarray(pos, np.float64)[:, None] * np.asarray(inv_freq, np.float32).astype(np.float64)
    c, s = np.cos(a)[:, None], np.sin(a)[:, None]
    lo = np.arange(half) * (2 if interleaved else 1)
    hi = lo + (1 if interleaved else half)
    y[..., lo], y[..., hi] = x[..., lo] * c - x[..., hi] * s, x[..., hi] * c + x[..., lo] * s
    return y


def attend(q, K, V, sees, sm_scale):
    """q [H, d], K, V [n, d] of the visible tokens' kv head, sees [n] bool -> (out [H, d], lse [H]), binary64."""
    q = np.asarray(q, np.float64)
    K, V = K[sees], V[sees]
    if len(K) == 0:
        return np.zeros_like(q), np.full(len(q), -np.inf)
    x = q @ K.T * sm_scale
    m = x.max(-1, keepdims=True)
    p = np.exp(x - m)
    z = p.sum(-1, keepdims=True)
    return p @ V / z, (m + np.log(z))[:, 0]
