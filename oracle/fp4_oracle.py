"""Plain 64-bit definitions of the microscaled 4-bit matrices (numpy; test infrastructure only).

Everything is decided in fp64, in which the quotients' comparisons are exact: a border between two
codes times a block scale has at most 7 significant bits.  Nothing here is shared with the library.
"""
from __future__ import annotations

import numpy as np

NV, MX = 0, 1
BLOCK = {NV: 16, MX: 32}
E2M1 = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6], dtype=np.float64)
E4M3 = np.array([m * 2.0 ** -9 for m in range(8)]
                + [(8 + m) * 2.0 ** (e - 10) for e in range(1, 16) for m in range(8)][:-1])


def nearest(v, grid):
    """Index of the nearest value of an ascending grid, of two as near the even one (saturating)."""
    hi = np.clip(np.searchsorted(grid, v), 1, len(grid) - 1)
    up, down = grid[hi] - v, v - grid[hi - 1]
    return np.where((up < down) | ((up == down) & (hi % 2 == 0)), hi, hi - 1)


def pow2_scale(x):
    """Smallest power of two g >= 2^-126 with max |x| <= 6 * 448 g; what is not finite left out."""
    a = np.abs(np.asarray(x, dtype=np.float64))
    a = float(a[np.isfinite(a)].max(initial=0.0))
    k = -126
    while a > 2688.0 * 2.0 ** k:
        k += 1
    return 2.0 ** k


def quantize(x, fmt, g=1.0):
    """x [rows, depth] -> (codes 0..15 [rows, blocks, B], scale codes [rows, blocks]), the depth padded
    with zeros to whole blocks.  g: the matrix's scale (NV)."""
    x = np.asarray(x, dtype=np.float64)
    R, D = x.shape
    B = BLOCK[fmt]
    p = np.zeros((R, -(-D // B) * B))
    if fmt == NV:  # x times fl32(1/g), rounded to fp32
        inv = float(np.float32(1.0) / np.float32(g))
        with np.errstate(over="ignore", invalid="ignore"):
            p[:, :D] = (x * inv).astype(np.float32)
    else:
        p[:, :D] = x
    p = p.reshape(R, -1, B)
    a = np.abs(p).max(-1)
    bad = ~np.isfinite(a)
    a = np.where(bad, 0.0, a)
    p = np.where(bad[..., None], 0.0, p)
    if fmt == NV:
        sc = nearest(np.minimum(a / 6.0, 448.0), E4M3)
        s = E4M3[sc]
        sc = np.where(bad, 0x7F, sc)
    else:
        e = np.frexp(np.where(a > 0, a, 1.0))[1] - 1  # a = m 2^e, 1 <= m < 2
        sc = np.where(a > 0, np.maximum(e - 2 + 127, 0), 0)
        s = 2.0 ** (sc - 127.0)
        sc = np.where(bad, 0xFF, sc)
    q = np.where(s[..., None] > 0, np.abs(p) / np.where(s > 0, s, 1.0)[..., None], 0.0)
    codes = nearest(q, E2M1) + 8 * np.signbit(p)
    return codes, sc


def scale_values(sc, fmt):
    sc = np.asarray(sc)
    if fmt == NV:
        return np.where(sc == 0x7F, np.nan, E4M3[np.minimum(sc, 126)])
    return np.where(sc == 0xFF, np.nan, 2.0 ** (sc - 127.0))


def values(codes, sc, fmt, depth, g=1.0):
    """code * s * g [rows, depth]: code * s is exact, its product with g (an fp32 number) is the one
    that the library rounds to fp32."""
    v = E2M1[codes & 7] * np.where(codes & 8, -1.0, 1.0) * scale_values(sc, fmt)[..., None]
    return v.reshape(v.shape[0], -1)[:, :depth] * float(np.float32(g))


def rounded(x, fmt, g=1.0):
    """The round trip of x [rows, depth] in 64 bits."""
    return values(*quantize(x, fmt, g), fmt, np.asarray(x).shape[1], g)


def pack(codes, sc, fmt, depth):
    """(values bytes [rows, D / 2], scale bytes [tiles, chunks, 512]) as the layout stores one matrix
    that is not ragged; scale bytes of rows past the last are 0 here and unspecified there."""
    R = codes.shape[0]
    B = BLOCK[fmt]
    D = -(-depth // 128) * 128
    c = np.zeros((R, D), dtype=np.uint8)
    c[:, :codes.shape[1] * B] = codes.reshape(R, -1)
    s = np.zeros((-(-R // 128), D // (4 * B), 512), dtype=np.uint8)
    for r in range(R):
        for b in range(sc.shape[1]):
            s[r // 128, b // 4, 16 * (r % 32) + 4 * (r // 32 % 4) + b % 4] = sc[r, b]
    return c[:, 0::2] | c[:, 1::2] << 4, s


def activate(y, act):
    from math import erf
    if act == 1:
        return np.maximum(y, 0.0)
    if act == 2:
        return y / (1.0 + np.exp(-y))
    if act == 3:
        return 0.5 * y * (1.0 + np.vectorize(erf)(y / np.sqrt(2.0)))
    return y
