"""Oracle of the rotary append and of the 4-bit cache (numpy, 64 bits).

TEST INFRASTRUCTURE ONLY.  Written from the definitions in include/resa.h
(resa_cache_q4_t, resa_rope_t), sharing no code with the CUDA library: group
scales and codes are found by searching the table of representable values.
"""
from __future__ import annotations

import numpy as np

E2M1 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
# e4m3 magnitudes of bytes 0 .. 126 (127 is NaN): exponent bias 7, 3 mantissa bits
E4M3 = np.array([(m / 8 * 2.0 ** -6) if e == 0 else (1 + m / 8) * 2.0 ** (e - 7)
                 for e in range(16) for m in range(8)][:127])


def nearest(x, table):
    """Index of the entry of the ascending table nearest to x >= 0; ties to the even index;
    values past the end take the last entry."""
    x = np.asarray(x, dtype=np.float64)
    hi = np.clip(np.searchsorted(table, x), 1, len(table) - 1)
    lo = hi - 1
    dl, dh = x - table[lo], table[hi] - x
    up = (dh < dl) | ((dh == dl) & (hi % 2 == 0))
    return np.where(up, hi, lo)


def bf16(x):
    """float64 -> float32 -> nearest bf16, as float64 (finite values)."""
    u = np.asarray(x, dtype=np.float32).view(np.uint32).astype(np.uint64)
    u = (u + 0x7fff + ((u >> 16) & 1)) & 0xffff0000
    return u.astype(np.uint32).view(np.float32).astype(np.float64)


def quantise(x, g):
    """x [..., d] (bf16 values) with heads' scales g broadcastable to [..., 1]: codes [..., d]
    (4-bit numbers) and group scale bytes [..., d / 16]."""
    x = np.asarray(x, dtype=np.float32)
    rg = np.float32(1) / np.asarray(g, dtype=np.float32)
    with np.errstate(over="ignore", invalid="ignore"):
        y = (x * rg).reshape(*x.shape[:-1], x.shape[-1] // 16, 16)
    a = np.where(np.isnan(y), np.float32(0), np.abs(y))
    s = nearest(np.minimum(a.max(-1) / np.float32(6), np.float32(1e30)), E4M3)
    t = E4M3[s][..., None]
    # nearest code: a / t against the table, compared as a against table * t (exact in 64 bits)
    code = np.zeros(a.shape, dtype=np.int64)
    mid = (E2M1[1:] + E2M1[:-1]) / 2
    for i, m in enumerate(mid):            # from code i to i + 1; ties to the even code
        code += (a >= m * t) if (i + 1) % 2 == 0 else (a > m * t)
    code = np.where(t > 0, code, 0)
    neg = (y < 0) & (t > 0)
    return (code + 8 * neg).reshape(x.shape).astype(np.uint8), s.astype(np.uint8)


def values(code, s):
    """c * s of codes [..., d] and scale bytes [..., d / 16]: float64, exact."""
    v = np.where(code >= 8, -E2M1[code & 7], E2M1[code & 7])
    return (v.reshape(*code.shape[:-1], code.shape[-1] // 16, 16) * E4M3[s][..., None]).reshape(code.shape)


def pack(code):
    return (code[..., 0::2] | (code[..., 1::2] << 4)).astype(np.uint8)


def unpack(b):
    return np.stack([b & 15, b >> 4], axis=-1).reshape(*b.shape[:-1], 2 * b.shape[-1])


def rotate(x, pos, inv_freq, rot, interleaved, mscale=1.0):
    """x [n, heads, d] float64 at positions pos [n]."""
    x = np.array(x, dtype=np.float64)
    if rot == 0:
        return x
    ang = np.asarray(pos, dtype=np.float64)[:, None] * np.asarray(inv_freq, dtype=np.float64)
    c, s = np.cos(ang)[:, None] * mscale, np.sin(ang)[:, None] * mscale
    i1, i2 = ((np.arange(0, rot, 2), np.arange(1, rot, 2)) if interleaved
              else (np.arange(rot // 2), np.arange(rot // 2, rot)))
    a, b = x[..., i1].copy(), x[..., i2].copy()
    x[..., i1] = a * c - b * s
    x[..., i2] = b * c + a * s
    return x


def attention(q, k, v, limit, scale):
    """q [rows, d] against k, v [n, d] (float64); row i sees the first limit[i] of them.  Returns
    the output, the log-sum-exp, sum p |v|, the largest sum |q k| of a row's keys and sum |v|."""
    x = q @ k.T * scale
    mag = (np.abs(q) @ np.abs(k).T * scale).max(-1, initial=0.0)
    x = np.where(np.arange(k.shape[0])[None] < np.asarray(limit)[:, None], x, -np.inf)
    m = x.max(-1, keepdims=True, initial=-np.inf)
    p = np.exp(x - np.where(np.isfinite(m), m, 0))
    z = p.sum(-1, keepdims=True)
    w = p / np.where(z > 0, z, 1)
    with np.errstate(divide="ignore"):
        lse = (np.where(np.isfinite(m), m, 0) + np.log(z))[:, 0]
    return w @ v, lse, w @ np.abs(v), mag, np.abs(v).sum(0)
