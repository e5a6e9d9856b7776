"""Oracle: the AdamW step, the norm of gradients, and the 8-bit form of the
moments, fp64 on the CPU.  TEST INFRASTRUCTURE ONLY (see the package docstring).

The 8-bit moments: blocks of 256 elements hold m and sqrt(v) as e4m3 values
times a scale, the block's largest magnitude / 448, rounded up with the chance
of the remainder; the chances come from Wellons' lowbias32 hash of place, step
and seed and the Numerical Recipes congruential sequence.
"""

from __future__ import annotations

import math

import numpy as np

BLOCK = 256
TOP = 448.0


def grad_norm(grads) -> float:
    return math.sqrt(math.fsum(float((np.asarray(g, dtype=np.float64) ** 2).sum()) for g in grads))


def step(p, g, m, v, t: int, lr, betas=(0.9, 0.999), eps=1e-8, decay=0.01, clip=1.0):
    """(p, m, v, change) after step t (counted from 1)."""
    p, g, m, v = (np.asarray(a, dtype=np.float64) for a in (p, g, m, v))
    g = g * clip
    m = betas[0] * m + (1.0 - betas[0]) * g
    v = betas[1] * v + (1.0 - betas[1]) * g * g
    change = lr / (1.0 - betas[0] ** t) * m / (np.sqrt(v / (1.0 - betas[1] ** t)) + eps)
    return p * (1.0 - lr * decay) - change, m, v, change


def lowbias32(z):
    z = np.asarray(z, dtype=np.uint32)
    z = z ^ (z >> np.uint32(16))
    z = z * np.uint32(0x7FEB352D)
    z = z ^ (z >> np.uint32(15))
    z = z * np.uint32(0x846CA68B)
    return z ^ (z >> np.uint32(16))


def chances(blocks, t: int, seed: int):
    """(for m, for v) [blocks, 256]: the part of a step that is added before rounding down, in (0, 1)."""
    with np.errstate(over="ignore"):
        key = lowbias32(np.uint32((seed + t * 0x9E3779B9) % (1 << 32)))
        place = (np.asarray(blocks, dtype=np.uint64)[:, None] * 32 + np.arange(32, dtype=np.uint64)) % (1 << 32)
        r = lowbias32(place.astype(np.uint32) ^ key)
        out = np.zeros((16,) + r.shape)
        for k in range(16):
            r = r * np.uint32(1664525) + np.uint32(1013904223)
            out[k] = ((r >> np.uint32(16)) * 16.0 + 8.0) / 2.0 ** 20
    u = np.moveaxis(out, 0, 2)      # [blocks, 32, 16]
    return u[:, :, :8].reshape(len(u), -1), u[:, :, 8:].reshape(len(u), -1)


def e4m3_step(x):
    """Distance of e4m3 values at |x|."""
    e = np.floor(np.log2(np.maximum(np.abs(x), 2.0 ** -6)))
    return 2.0 ** (e - 3)


def encode(x, u, positive: bool):
    """(codes, scales, distance of each value from where it would be rounded the other way, in steps) of blocks
    x [n, 256]; positive: codes of positive values stay at least 2^-9."""
    scale = np.abs(x).max(1) / TOP
    y = np.abs(x) / np.where(scale > 0, scale, 1.0)[:, None]
    s = e4m3_step(y)
    q = np.floor(y / s + u)
    near = np.minimum(y / s + u - q, q + 1 - (y / s + u))
    q = np.minimum(q * s, TOP)
    if positive:
        q = np.where(y > 0, np.maximum(q, 2.0 ** -9), 0.0)
    return np.copysign(q, x), scale, near
