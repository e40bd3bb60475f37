"""float64 definitions of what a layer does around the striped pool: the rotary
turn of queries and keys, 4-bit rows, and attention with modified scores.

TEST INFRASTRUCTURE ONLY -- see the package docstring.

Readings: a pair (u, v) at angle a becomes (u cos a - v sin a, v cos a + u sin a);
pairs are (i, i + r/2) or (2i, 2i + 1) of the r rotated values.  A 4-bit row
(E2M1: sign, 2 exponent bits with bias 1, 1 mantissa bit) has one E4M3 scale
per 16 values, the E4M3 value nearest to max |x / descale| / 6; its codes are
the E2M1 values nearest to (x / descale) / scale, ties to the even code,
magnitudes past 6 at 6, all quotients rounded to float32; a block whose scale
is 0 is zeros, and a NaN in a block gives the scale's NaN code.  Scores are
capped first, then take the distance term.
"""

from __future__ import annotations

import numpy as np

from .reference import NEG_INF, e4m3_value

ROPE_HALVES, ROPE_PAIRS = 0, 1


def rotate(x, positions, cos_sin, begin: int, style: int):
    """Rows x [T, H, D] (float64) turned by their positions' angles."""
    y = np.array(x, dtype=np.float64, copy=True)
    r = cos_sin.shape[1]
    for t, n in enumerate(positions):
        if n < 0:
            continue
        for i in range(r // 2):
            a, b = (begin + i, begin + i + r // 2) if style == ROPE_HALVES else (begin + 2 * i, begin + 2 * i + 1)
            c, s = float(cos_sin[n, i]), float(cos_sin[n, r // 2 + i])
            u, v = x[t, :, a], x[t, :, b]
            y[t, :, a] = u * c - v * s
            y[t, :, b] = v * c + u * s
    return y


def e2m1_value(code: int) -> float:
    """Value of a 4-bit E2M1 code: (1 + m/2) 2^(e-1), or m/2 for e = 0."""
    sign = -1.0 if code & 8 else 1.0
    e, m = (code >> 1) & 3, code & 1
    return sign * (m / 2.0 if e == 0 else (1.0 + m / 2.0) * 2.0 ** (e - 1))


def _nearest(vals, a):
    """Index of the value of the increasing list nearest to each a >= 0 (ties to
    the even index; past the last: the last)."""
    vals = np.asarray(vals, dtype=np.float64)
    a = np.asarray(a, dtype=np.float64)
    lo = np.clip(np.searchsorted(vals, a, side="right") - 1, 0, len(vals) - 1)
    hi = np.minimum(lo + 1, len(vals) - 1)
    d_lo, d_hi = a - vals[lo], vals[hi] - a
    up = (d_hi < d_lo) | ((d_hi == d_lo) & (lo % 2 == 1))
    return np.where(up & (hi > lo), hi, lo)


def e2m1_encode(x):
    """Nearest E2M1 codes (ties to the even code, saturated at 6)."""
    x = np.asarray(x, dtype=np.float64)
    code = _nearest([e2m1_value(c) for c in range(8)], np.abs(x))
    return (code | np.where(np.signbit(x), 8, 0)).astype(np.uint8)


def fp4_quantize(x, descale: float):
    """Codes [..., D] (one a value, unpacked) and scale codes [..., D / 16] of
    float32 rows."""
    x = np.asarray(x, dtype=np.float32)
    with np.errstate(all="ignore"):
        v = (x / np.float32(descale)).astype(np.float32).reshape(-1, 16)
        bad = np.isnan(v).any(axis=1)
        top = np.where(bad, 0, np.abs(v).max(axis=1)).astype(np.float32) / np.float32(6)
        vals = np.array([e4m3_value(c) for c in range(0x7F)])
        scales = _nearest(vals, top)
        s = vals[scales].astype(np.float32)[:, None]
        live = (s > 0) & ~bad[:, None]
        codes = np.where(live, e2m1_encode(np.where(live, v / np.where(live, s, 1), 0)), 0)
    scales = np.where(bad, 0x7F, scales).astype(np.uint8)
    return codes.astype(np.uint8).reshape(x.shape), scales.reshape(*x.shape[:-1], x.shape[-1] // 16)


def fp4_dequantize(codes, scales, descale: float):
    """float64 values of stored codes and scales."""
    t = np.array([e2m1_value(c) for c in range(16)])
    s = np.array([e4m3_value(c) for c in range(256)])
    v = t[np.asarray(codes)].reshape(-1, 16) * s[np.asarray(scales).reshape(-1)][:, None]
    return v.reshape(np.shape(codes)) * float(np.float32(descale))


def fp4_pack(codes):
    """Bytes [..., D / 2] of unpacked codes: even value in the low half."""
    c = np.asarray(codes, dtype=np.uint8)
    return c[..., 0::2] | (c[..., 1::2] << 4)


def modified_attention(q, K, V, scale: float, qpos: int, kpos, softcap: float = 0.0, slopes=None):
    """One query token [Hq, D] at position qpos over keys at positions kpos:
    (O [Hq, Dv], LSE [Hq], A [Hq, Dv] = the weights applied to |V|, B [Hq, Dv] =
    sum of |V| over the sum of exp(s - max s))."""
    Hq, (m, Hkv), Dv = q.shape[0], K.shape[:2], V.shape[2]
    O, A, B = np.zeros((Hq, Dv)), np.zeros((Hq, Dv)), np.zeros((Hq, Dv))
    L = np.full((Hq,), NEG_INF)
    if m == 0:
        return O, L, A, B
    for h in range(Hq):
        kh = h // (Hq // Hkv)
        s = scale * (K[:, kh, :] @ q[h])
        if softcap:
            s = softcap * np.tanh(s / softcap)
        if slopes is not None:
            s = s + float(slopes[h]) * (np.asarray(kpos, np.float64) - qpos)
        mx = s.max()
        w = np.exp(s - mx)
        z = w.sum()
        O[h], A[h], L[h] = (w @ V[:, kh]) / z, (w @ np.abs(V[:, kh])) / z, mx + np.log(z)
        B[h] = np.abs(V[:, kh]).sum(axis=0) / z
    return O, L, A, B
