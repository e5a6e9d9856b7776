"""Oracle: positions of packed segments, and rotary positions of queries and
keys with the RMS norm before them and its gradient, fp64 on the CPU.  TEST
INFRASTRUCTURE ONLY (see the package docstring).

Per head vector x [D], in fp64 from the inputs as handed to the kernels:

    r = 1 / sqrt(mean x^2 + eps)  over the head ("head") or all heads of the
        token ("token");  z = x r w  (no norm: z = x)
    pair i of the first R features, angle t_i = pos[axis(i)] freq_i:
        (a, b) -> gain (a cos t - b sin t, a sin t + b cos t)

Angles are reduced in Python integers: freq_i / 2 pi is taken as an exact
fraction, so that far positions lose nothing.  The gradient turns the
upstream gradient back and applies the norm's:

    dx = r (g w - xh mean(g w xh)),  xh = x r,  dw = sum g xh
"""

from __future__ import annotations

import math
from fractions import Fraction

import numpy as np

from .adaln import _f64

# pi to 60 digits
_PI = Fraction("3.14159265358979323846264338327950288419716939937510582097494")


def positions(seg_frames, tokens_per_frame: int, L: int, axes: int = 1, row_width: int | None = None) -> np.ndarray:
    """int32 [B, L, axes]: position of each token inside its segment, token by token."""
    frames = np.asarray(seg_frames)
    out = np.zeros((frames.shape[0], L, axes), np.int32)
    for b, row in enumerate(frames):
        p = 0
        for f in row:
            for i in range(int(f) * tokens_per_frame):
                frame, slot = divmod(i, tokens_per_frame)
                out[b, p] = [[i], [frame, slot], [frame, slot // (row_width or 1), slot % (row_width or 1)]][axes - 1]
                p += 1
    return out


def rotary_angles(pos, freqs, sections) -> np.ndarray:
    """Angles in [0, 2 pi) of int positions [B, L, axes]: [B, L, R/2].  freqs: radians per position."""
    pos = np.asarray(pos)
    axis = np.repeat(np.arange(len(sections)), sections)
    out = np.empty(pos.shape[:2] + (len(freqs),))
    for i, f in enumerate(freqs):
        turns = Fraction(f) / (2 * _PI)
        col = pos[..., axis[i]]
        values = {int(v): float((int(v) * turns) % 1) * 2.0 * math.pi for v in np.unique(col)}
        out[..., i] = np.vectorize(values.__getitem__, otypes=[np.float64])(col)
    return out


def _turn(x, angle, R, layout, gain):
    c, s = gain * np.cos(angle)[:, :, None], gain * np.sin(angle)[:, :, None]
    out = x.copy()
    first, second = (slice(0, R // 2), slice(R // 2, R)) if layout == "half" else (slice(0, R, 2), slice(1, R, 2))
    a, b = x[..., first], x[..., second]
    out[..., first] = a * c - b * s
    out[..., second] = a * s + b * c
    return out


def _rms(x, norm, eps):
    ax = (2, 3) if norm == "token" else 3
    return 1.0 / np.sqrt((x * x).mean(axis=ax, keepdims=True) + eps), ax


def _weight(w, x, norm):
    w = np.ones(x.shape[3]) if w is None else _f64(w)
    return w.reshape(x.shape[2:]) if norm == "token" and w.size != x.shape[3] else w


def rotary_fwd(x, pos, freqs, sections, layout="half", gain=1.0, norm=None, weight=None, eps=1e-6):
    x = _f64(x)
    if norm:
        x = x * _rms(x, norm, eps)[0] * _weight(weight, x, norm)
    return _turn(x, rotary_angles(pos, freqs, sections), 2 * len(freqs), layout, gain)


def rotary_bwd(dout, pos, freqs, sections, layout="half", gain=1.0, norm=None, x=None, weight=None, eps=1e-6):
    """(dx, dweight or None, sum of the magnitudes that dweight adds or None)."""
    g = _turn(_f64(dout), -rotary_angles(pos, freqs, sections), 2 * len(freqs), layout, gain)
    if not norm:
        return g, None, None
    x = _f64(x)
    r, ax = _rms(x, norm, eps)
    xh = x * r
    over = (0, 1) if norm == "token" else (0, 1, 2)
    dw, mag = (g * xh).sum(axis=over).ravel(), np.abs(g * xh).sum(axis=over).ravel()
    g = g * _weight(weight, x, norm)
    return r * (g - xh * (g * xh).mean(axis=ax, keepdims=True)), dw, mag
