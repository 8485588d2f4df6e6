"""Plain numpy reference of the paged key/value cache (include/q4.h) for the tests: the
layout, the quantisers as single fp32 operations, and attention in fp64."""
from __future__ import annotations

import numpy as np

INT8, INT4 = 0, 1


def row_bytes(fmt, D):
    return D if fmt == INT8 else D // 2


def scale_bytes(fmt):
    return 2 if fmt == INT8 else 4


def block_bytes(fmt, D):
    return 32 * (row_bytes(fmt, D) + scale_bytes(fmt))


def place(fmt, D, r, b):
    """Offset of byte b of code row r among the K (or V) codes of a block."""
    rb = row_bytes(fmt, D)
    line, piece, rest = (r * rb + b) // 128, (r * rb + b) % 128 // 16, b % 16
    key = {128: r & 7, 64: r & 6, 32: (r >> 1) & 2}[rb]
    return line * 128 + (piece ^ key) * 16 + rest


def quantise(x, fmt):
    """Rows x fp32 [n, D] -> (code bytes uint8 [n, row bytes], scale bytes uint8 [n, scale bytes])."""
    x = np.asarray(x, np.float32)
    n, D = x.shape
    bad = ~np.isfinite(x).all(1)
    x = np.where(bad[:, None], np.float32(0), x)
    top = np.float32(65504)
    with np.errstate(all="ignore"):
        if fmt == INT8:
            s = np.minimum(np.abs(x).max(1) / np.float32(127), top).astype(np.float16)
            sf = s.astype(np.float32)[:, None]
            c = np.where(sf > 0, np.clip(np.rint(x / sf), -127, 127), 0).astype(np.int8).view(np.uint8)
            info = s.view(np.uint16)[:, None].copy()
        else:
            lo, hi = x.min(1), x.max(1)
            s = np.minimum((hi - lo) / np.float32(15), top).astype(np.float16)
            m = np.clip(lo, -top, top).astype(np.float16)
            sf, mf = s.astype(np.float32)[:, None], m.astype(np.float32)[:, None]
            q = np.where(sf > 0, np.clip(np.rint((x - mf) / sf), 0, 15), 0).astype(np.uint8)
            c = q[:, 0::2] | (q[:, 1::2] << 4)
            info = np.stack((s.view(np.uint16), m.view(np.uint16)), 1)
    info[bad] = 0x7FFF
    return c, np.ascontiguousarray(info).view(np.uint8)


def write(cache, slots, k, v, fmt, page):
    """Quantise rows k, v fp32 [n, H, D] into the slots of a cache (uint8 array, changed)."""
    n, H, D = k.shape
    rb, sb = row_bytes(fmt, D), scale_bytes(fmt)
    places = np.array([[place(fmt, D, r, b) for b in range(rb)] for r in range(16)])
    for x, at, info_at in ((k, 0, 32 * rb), (v, 16 * rb, 32 * rb + 16 * sb)):
        codes, info = quantise(x.reshape(n * H, D), fmt)
        codes, info = codes.reshape(n, H, rb), info.reshape(n, H, sb)
        for i, slot in enumerate(slots):
            if not 0 <= slot < cache.shape[0] * page:
                continue
            blk = cache[slot // page, :, slot % page // 16]
            r = slot % 16
            blk[:, at + places[r]] = codes[i]
            blk[:, info_at + sb * r:info_at + sb * (r + 1)] = info[i]


def read(cache, pages, length, fmt, D):
    """(k, v) fp32 [length, H, D] of the first tokens of a list of pages: the exact value, or
    (int4) that of one fp32 multiply-add.  A page outside the cache gives NaN rows (marker)."""
    page = cache.shape[2] * 16
    H = cache.shape[1]
    rb, sb = row_bytes(fmt, D), scale_bytes(fmt)
    places = np.array([[place(fmt, D, r, b) for b in range(rb)] for r in range(16)])
    out = np.zeros((2, length, H, D), np.float32)
    pos = np.arange(length)
    pg = np.asarray(pages)[pos // page] if length else np.zeros(0, int)
    ok = (pg >= 0) & (pg < cache.shape[0])
    blk = cache[np.where(ok, pg, 0), :, pos % page // 16]              # [length, H, bytes]
    r = pos % 16
    for i, (at, info_at) in enumerate(((0, 32 * rb), (16 * rb, 32 * rb + 16 * sb))):
        codes = np.take_along_axis(blk, (at + places[r])[:, None, :].repeat(H, 1), 2) if length else \
            np.zeros((0, H, rb), np.uint8)
        idx = info_at + sb * r[:, None] + np.arange(sb)
        info = np.ascontiguousarray(np.take_along_axis(blk, idx[:, None, :].repeat(H, 1), 2)).view(np.float16)
        info = info.astype(np.float32)
        with np.errstate(all="ignore"):
            if fmt == INT8:
                x = codes.view(np.int8).astype(np.float32) * info
            else:
                c = np.stack((codes & 15, codes >> 4), -1).reshape(length, H, D).astype(np.float64)
                x = (c * info[..., :1] + info[..., 1:]).astype(np.float32)
        out[i] = x
        out[i][~ok] = np.nan
    return out[0], out[1], ok


def attention(q, k, v, ok, limits, scale):
    """fp64 attention of one sequence.  q [T, Hq, D]; k, v [n, H, D]; ok [n]: tokens attended to;
    limits [T].  Returns (out, sum of p |v|) [T, Hq, D]."""
    T, Hq, D = q.shape
    H = k.shape[1]
    out = np.zeros((T, Hq, D))
    mag = np.zeros((T, Hq, D))
    q, k, v = q.astype(np.float64), k.astype(np.float64), v.astype(np.float64)
    pos = np.arange(k.shape[0])
    for t in range(T):
        use = ok & (pos < limits[t])
        if not use.any():
            continue
        for h in range(Hq):
            kk, vv = k[use, h * H // Hq], v[use, h * H // Hq]
            s = kk @ q[t, h] * scale
            p = np.exp(s - s.max())
            p /= p.sum()
            out[t, h] = p @ vv
            mag[t, h] = p @ np.abs(vv)
    return out, mag
