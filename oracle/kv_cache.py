"""Oracle of the paged cache's writers and of its 4-bit form (test
infrastructure only). The rotation of an appended row and the 4-bit codes are
defined down to the roundings, so that what is written is compared bit for bit;
the decoding step is fp64."""
from __future__ import annotations

import numpy as np

from .attention import NEG_INF
from .norm_rope import _pairs

GROUP = 64


def to_bf16(x):
    """float64 or float32 values (the latter exactly representable in float64)
    rounded to bf16, ties to even, as float64; NaN and infinities as they are."""
    x = np.asarray(x, np.float64)
    m, e = np.frexp(np.where(np.isfinite(x), x, 0.0))
    unit = np.exp2(np.maximum(e - 8, -133).astype(np.float64))  # 8 significant bits, subnormals from 2^-126 down
    y = np.round(np.where(np.isfinite(x), x, 0.0) / unit) * unit
    y = np.where(np.abs(y) >= 2.0 ** 128, np.copysign(np.inf, y), y)
    return np.where(np.isfinite(x), y, x)


def rotated(x, cos, sin, positions, interleaved):
    """bf16 rows x [T, H, d] (as float64) turned, every product and sum in
    fp32, the result in bf16 (as float64)."""
    x32 = np.asarray(x, np.float32)
    y = x32.copy()
    c, s = (np.asarray(t, np.float32)[positions][:, None, :] for t in (cos, sin))
    a, b = _pairs(2 * c.shape[-1], interleaved)
    y[..., a] = to_bf16(x32[..., a] * c - x32[..., b] * s)
    y[..., b] = to_bf16(x32[..., b] * c + x32[..., a] * s)
    return y.astype(np.float64)


def quantise_q4(x):
    """bf16 rows [..., d] (as float64): codes [..., d] (integers) and (s, z) [..., d / 64, 2]."""
    x = np.asarray(x, np.float64)
    g = x.reshape(*x.shape[:-1], x.shape[-1] // GROUP, GROUP)
    with np.errstate(all="ignore"):
        z = np.min(g, -1)
        width = (np.max(g, -1).astype(np.float32) - z.astype(np.float32)).astype(np.float64)
        s = to_bf16(width / 15)
        s = np.where(s < 2.0 ** -126, 0.0, s)
        bad = ~np.isfinite(s)
        s, z = np.where(bad, np.nan, s), np.where(bad, np.nan, z)
        t = (g.astype(np.float32) - z[..., None].astype(np.float32)).astype(np.float64)
        code = np.where((s > 0)[..., None], np.round(t / s[..., None]), 0.0)
    return np.clip(code, 0, 15).reshape(x.shape).astype(np.int64), np.stack((s, z), -1)


def held_q4(codes, scales):
    """What codes [..., d] with (s, z) [..., d / 64, 2] stand for."""
    per = np.repeat(np.asarray(scales, np.float64), GROUP, -2)
    return per[..., 1] + per[..., 0] * codes


def held_q4_bf16(codes, scales):
    """held_q4 rounded once to bf16, however far apart z and s are: a sum that
    fp64 rounded is first taken to its odd neighbour, which no bf16 tie is."""
    per = np.repeat(np.asarray(scales, np.float64), GROUP, -2)
    with np.errstate(invalid="ignore"):
        z, p = per[..., 1], per[..., 0] * codes
        x = z + p
        part = x - z
        err = (z - (x - part)) + (p - part)
        even = (np.ascontiguousarray(x).view(np.int64) & 1) == 0
        towards = np.nextafter(x, np.copysign(np.inf, err))
        return to_bf16(np.where(even & np.isfinite(err) & (err != 0), towards, x))


def unpack_codes(packed):
    """uint8 [..., d / 2] -> integers [..., d]."""
    p = np.asarray(packed).astype(np.int64)
    return np.stack((p & 15, p >> 4), -1).reshape(*p.shape[:-1], 2 * p.shape[-1])


def q4_decode_forward(q, k, v, seq_lens, scale):
    """q [B, n, H, d]; k and v: a list of [L_b, Hk, d] per sequence. Returns
    O [B, n, H, d], LSE [B, n, H] and A = sum of P |V|."""
    q = np.asarray(q, np.float64)
    B, n, H, d = q.shape
    o, a, lse = np.zeros(q.shape), np.zeros(q.shape), np.full((B, n, H), NEG_INF)
    for b in range(B):
        Hk = k[b].shape[1]
        for i in range(n):
            seen = int(seq_lens[b]) - n + i + 1
            if seen <= 0:
                continue
            for h in range(H):
                j = h // (H // Hk)
                x = scale * (k[b][:seen, j] @ q[b, i, h])
                m = np.max(x)
                p = np.exp(x - m)
                t = np.sum(p)
                o[b, i, h], a[b, i, h] = p @ v[b][:seen, j] / t, p @ np.abs(v[b][:seen, j]) / t
                lse[b, i, h] = m + np.log(t)
    return o, lse, a
