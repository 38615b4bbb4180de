"""Microscaled 4-bit rows and the norm/residual step, in plain float64.

Test infrastructure; shares no code with the CUDA library.  Values, scales
and the products of a scale with a border between two codes are exact in
float64, so nearest-value decisions here are those of real arithmetic.
"""
from __future__ import annotations

import numpy as np

MX, NV = 0, 1
BLOCK = {MX: 32, NV: 16}
E2M1 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
E4M3 = np.array([(b & 7) * 2.0 ** -9 if b < 8 else (1 + (b & 7) / 8) * 2.0 ** ((b >> 3) - 7) for b in range(127)])


def nearest(table: np.ndarray, a: np.ndarray) -> np.ndarray:
    """Index of the table value nearest to a >= 0; ties to the even index."""
    hi = np.minimum(np.searchsorted(table, a), len(table) - 1)
    lo = np.maximum(hi - 1, 0)
    dlo, dhi = a - table[lo], table[hi] - a
    return np.where((dlo < dhi) | ((dlo == dhi) & (lo % 2 == 0)), lo, hi)


def quant(x, fmt: int):
    """x [R, K] -> (codes [R, K/2] uint8, scale bytes [R, K/B] uint8, row scale [R])."""
    x = np.asarray(x, np.float64)
    R, K = x.shape
    B = BLOCK[fmt]
    v = x.reshape(R, K // B, B)
    a = np.abs(v)
    bad = ~np.isfinite(a).all(-1)
    amax = np.where(bad, 0.0, np.where(np.isfinite(a), a, 0.0).max(-1))
    S = np.ones(R)
    if fmt == MX:
        _, ex = np.frexp(amax)                       # amax = m 2^ex, 0.5 <= m < 1
        e = np.where(amax > 0, np.maximum(ex - 1 - 2, -127), 0)
        byte, s = e + 127, np.ldexp(1.0, e)
    else:
        top = amax.max(-1)
        for r in range(R):
            if top[r] > 0:
                e = -126
                while top[r] > 2688.0 * 2.0 ** e:
                    e += 1
                S[r] = 2.0 ** e
        byte = nearest(E4M3, amax / (6.0 * S[:, None]))
        s = E4M3[byte]
    scale = (s * S[:, None])[..., None]
    with np.errstate(invalid="ignore", divide="ignore"):
        mag = nearest(E2M1, np.where(scale > 0, np.where(np.isfinite(a), a, 0.0) / np.where(scale > 0, scale, 1.0), 0.0))
    code = np.where(scale > 0, mag + 8 * np.signbit(v), 0)
    code = np.where(bad[..., None], 0, code).astype(np.uint8).reshape(R, K)
    byte = np.where(bad, 255 if fmt == MX else 127, byte).astype(np.uint8)
    return code[:, 0::2] | (code[:, 1::2] << 4), byte, S


def scale_value(byte, fmt: int) -> np.ndarray:
    b = np.asarray(byte).astype(np.int64)
    if fmt == MX:
        return np.where(b == 255, np.nan, np.ldexp(1.0, b - 127))
    return np.where((b & 127) == 127, np.nan, E4M3[np.minimum(b & 127, 126)])


def unpack(codes) -> np.ndarray:
    """[R, K/2] bytes -> signed E2M1 values [R, K]."""
    c = np.asarray(codes)
    c = np.stack([c & 15, c >> 4], -1).reshape(c.shape[0], -1)
    return np.where(c & 8, -1.0, 1.0) * E2M1[c & 7]


def values(codes, byte, row_scale, fmt: int) -> np.ndarray:
    """The numbers that codes and scales stand for, [R, K]."""
    q = unpack(codes)
    R, K = q.shape
    v = (q.reshape(R, K // BLOCK[fmt], -1) * scale_value(byte, fmt)[..., None]).reshape(R, K)
    return v if row_scale is None else v * np.asarray(row_scale, np.float64)[:, None]


def tile_scales(byte, fmt: int) -> np.ndarray:
    """Scale bytes [R, K/B] -> the tiled buffer, padding zero."""
    R, C = byte.shape
    rt, ct = (R + 127) // 128, (C + 3) // 4
    out = np.zeros(rt * ct * 512, np.uint8)
    r, c = np.meshgrid(np.arange(R), np.arange(C), indexing="ij")
    out[((r // 128) * ct + c // 4) * 512 + 16 * (r % 32) + 4 * ((r % 128) // 32) + c % 4] = byte
    return out


def norm_residual(r, y=None, post_norm=False, post_w=None, gate=None, pre_w=None, res_scale=1.0, eps=1e-6,
                  w_offset=0.0):
    """(r', h) in float64."""
    def norm(v, w):
        v = v / np.sqrt((v * v).mean(-1, keepdims=True) + eps)
        return v if w is None else v * (w_offset + np.asarray(w, np.float64))

    r = np.asarray(r, np.float64)
    if y is not None:
        u = np.asarray(y, np.float64)
        if post_norm:
            u = norm(u, post_w)
        if gate is not None:
            u = u * np.asarray(gate, np.float64)
        r = res_scale * r + u
    return r, norm(r, pre_w)
