"""Plain numpy restatement of MXFP4 (OCP microscaling formats, version 1.0):
quantisation, decoding, scale tiles and the product, in 64 bits."""
from __future__ import annotations

import math

import numpy as np

MAGNITUDES = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def quantize(x):
    """x (rows, K) float64 -> codes (rows, KB, 32) and scale bytes (rows, KB), element by element."""
    rows, K = x.shape
    KB = -(-K // 32)
    codes = np.zeros((rows, KB, 32), np.uint8)
    scales = np.zeros((rows, KB), np.uint8)
    for r in range(rows):
        for b in range(KB):
            blk = x[r, 32 * b:32 * b + 32]
            if not np.all(np.isfinite(blk)):
                scales[r, b] = 255
                continue
            m = float(np.max(np.abs(blk)))
            e = -127 if m == 0 else max(-127, min(127, math.frexp(m)[1] - 3))
            scales[r, b] = e + 127
            for i, v in enumerate(blk):
                a = abs(float(v)) * 2.0 ** -e
                d = np.abs(MAGNITUDES - a)
                near = np.flatnonzero(d == d.min())
                c = int(near[0]) if len(near) == 1 else int(near[near % 2 == 0][0])
                codes[r, b, i] = c + (8 if math.copysign(1.0, float(v)) < 0 else 0)
    return codes, scales


def pack(codes):
    rows, KB, _ = codes.shape
    c = codes.reshape(rows, KB * 16, 2)
    return (c[:, :, 0] | (c[:, :, 1] << 4)).astype(np.uint8)


def unpack(q):
    rows, nb = q.shape
    return np.stack([q & 15, q >> 4], axis=2).reshape(rows, nb // 16, 32)


def tile_scales(scales, fill=0):
    rows, KB = scales.shape
    RB, KT = -(-rows // 128), -(-KB // 4)
    out = np.full((RB, KT, 512), fill, np.uint8)
    for r in range(rows):
        for b in range(KB):
            out[r // 128, b // 4, (r % 32) * 16 + (r % 128 // 32) * 4 + b % 4] = scales[r, b]
    for r in range(rows):          # blocks past K: zero
        for b in range(KB, 4 * KT):
            out[r // 128, b // 4, (r % 32) * 16 + (r % 128 // 32) * 4 + b % 4] = 0
    return out


def row_scales(tiles, rows, KB):
    out = np.zeros((rows, KB), np.uint8)
    for r in range(rows):
        for b in range(KB):
            out[r, b] = tiles[r // 128, b // 4, (r % 32) * 16 + (r % 128 // 32) * 4 + b % 4]
    return out


def decode(codes, scales):
    """Values (rows, KB * 32) in float64."""
    mag = MAGNITUDES[codes & 7]
    val = np.where(codes >= 8, -mag, mag)
    s = np.where(scales == 255, np.nan, np.ldexp(1.0, scales.astype(np.int64) - 127))
    return (val * s[:, :, None]).reshape(codes.shape[0], -1)


def product(a, w, relu):
    """C in float64 and the sum of the terms' magnitudes, for decoded operands."""
    c = a @ w.T
    mag = np.abs(a) @ np.abs(w).T
    return (np.where(c > 0, c, 0.0) if relu else c), mag


def product_tolerance(ref, mag, K):
    """One rounding to fp16 (half a step: 2^-11 relative, 2^-25 below the normal
    range) and the fp32 sum: products of two E2M1 values and powers of two are
    exact, one addition per MMA step of 64 elements and per slice of K, each
    off by at most two steps of fp32 (2^-22) of the sum of magnitudes."""
    return 2.0 ** -11 * np.abs(ref) + 2.0 ** -25 + (K / 64 + 16) * 2.0 ** -22 * mag
