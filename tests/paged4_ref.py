"""Rotary positions and the paged 4-bit cache in numpy, for the tests: plain
code from the definitions in include/kvq.h."""
import numpy as np

import paged_ref

MOST = 65408.0  # the largest magnitude that is stored
GROUP = 32


def frequencies(dim, base=10000.0, factor=1.0, original=0.0, low=1.0, high=32.0):
    """Radians a position of each pair."""
    f = base ** (-2.0 * np.arange(dim // 2) / dim)
    keep = np.zeros_like(f)
    if original:
        keep = np.clip((original * f / (2 * np.pi) - low) / (high - low), 0.0, 1.0)
    return f * keep + f / factor * (1 - keep)


def angles(positions, turns, magnitude=1.0):
    """float64 [T][n][2]: the part of a turn by whole-number arithmetic."""
    out = np.zeros((len(positions), len(turns), 2))
    for t, p in enumerate(positions):
        for i, f in enumerate(turns):
            part = (int(p) * int(f)) % (1 << 64)
            if part >= 1 << 63:
                part -= 1 << 64
            a = part * (2 * np.pi / 2.0 ** 64)
            out[t, i] = magnitude * np.cos(a), magnitude * np.sin(a)
    return out


def rotate(x, ang, interleaved):
    """float32 x [T][heads][D] turned by float32 angles: products and sums rounded
    to float32, one at a time."""
    x, ang = x.astype(np.float32), ang.astype(np.float32)
    r = 2 * ang.shape[1]
    a, b = (slice(0, r, 2), slice(1, r, 2)) if interleaved else (slice(0, r // 2), slice(r // 2, r))
    c, s = ang[:, None, :, 0], ang[:, None, :, 1]
    out = x.copy()
    out[..., a] = x[..., a] * c - x[..., b] * s
    out[..., b] = x[..., b] * c + x[..., a] * s
    return out


def quantize(x):
    """x: fp16-valued [..., D].  (codes [..., D], step and minimum [..., D / 32])."""
    x = np.asarray(x, np.float64)
    x = np.clip(np.where(np.isnan(x), 0.0, x), -MOST, MOST).astype(np.float16).astype(np.float32)
    g = x.reshape(*x.shape[:-1], -1, GROUP)
    mn, mx = g.min(-1), g.max(-1)
    step = ((mx - mn) / np.float32(15)).astype(np.float16)
    s = step.astype(np.float32)[..., None]
    q = (g - mn[..., None]) / np.where(s > 0, s, np.float32(1))
    codes = np.where(s > 0, np.clip(np.rint(q), 0, 15), 0).astype(np.uint8)
    return codes.reshape(x.shape), step, (mn + np.float32(0)).astype(np.float16)


def pack(codes, key):
    """Bytes [..., D / 2] of codes [..., D]: bit by bit from the words' definition."""
    D = codes.shape[-1]
    words = np.zeros((*codes.shape[:-1], D // 8), np.uint32)
    for c in range(D):
        i, j = divmod(c, 8)
        at = 4 * (j // 2) + 16 * (j % 2) if key else 4 * j
        words[..., i] |= codes[..., c].astype(np.uint32) << np.uint32(at)
    return words.astype("<u4").view(np.uint8)


def unpack(data, key):
    words = np.ascontiguousarray(data).view("<u4")
    codes = np.zeros((*words.shape[:-1], words.shape[-1] * 8), np.uint8)
    for c in range(codes.shape[-1]):
        i, j = divmod(c, 8)
        at = 4 * (j // 2) + 16 * (j % 2) if key else 4 * j
        codes[..., c] = (words[..., i] >> np.uint32(at)) & 15
    return codes


def values(codes, step, mn):
    """float64 of the fp16 numbers that codes stand for."""
    g = codes.reshape(*codes.shape[:-1], -1, GROUP).astype(np.float64)
    v = g * step.astype(np.float64)[..., None] + mn.astype(np.float64)[..., None]
    return v.astype(np.float16).astype(np.float64).reshape(codes.shape)


def attention(q, k, v, table, cu, seq, ps, scale, window, log2, half_step):
    """(out, bound) of all new tokens over pages of values k, v [pages][H][ps][D];
    the bound is paged_ref.row's for values without page scales."""
    R = q.shape[1] // k.shape[1]
    out, bound = np.zeros(q.shape), np.full(q.shape, 2.0 ** -25)
    for b in range(len(seq)):
        n = int(cu[b + 1] - cu[b])
        t = np.arange(seq[b])
        pg, r = table[b][t // ps], t % ps
        for h in range(k.shape[1] if n else 0):
            kk, vv = k[pg, h, r], v[pg, h, r]
            for j in range(n):
                pos = int(seq[b]) - n + j
                lo = max(0, pos - window + 1) if window else 0
                if pos < lo:
                    continue
                s = slice(lo, pos + 1)
                for hq in range(h * R, h * R + R):
                    out[cu[b] + j, hq], bound[cu[b] + j, hq], _ = paged_ref.row(
                        q[cu[b] + j, hq], kk[s], vv[s], np.ones(pos + 1 - lo), scale, log2, half_step)
    return out, bound
