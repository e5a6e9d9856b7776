"""Oracle: the gated residual with the norms on both sides of the block, and
its gradient, fp64 on the CPU.  TEST INFRASTRUCTURE ONLY (see the package
docstring).

Per token with modulation row s (id >= 0):

    u     = h, or post(h) w2
    x_out = alpha x + gate_s u
    y     = (norm(x_out) w + b)(1 + scale_s) + shift_s

norm, post: (v - mean) / sqrt(var + eps) ("layer") or v / sqrt(mean v^2 +
eps) ("rms").  Padding (id < 0): x_out = x, y = 0; backward dx = dx_out,
dh = 0 and no part in any sum.  The backward takes x_out as its input.
"""

from __future__ import annotations

import numpy as np

from .adaln import _f64


def _opt(t):
    return None if t is None else _f64(t)


def _norm(v, kind, eps):
    c = v - v.mean(axis=1, keepdims=True) if kind == "layer" else v
    r = 1.0 / np.sqrt((c * c).mean(axis=1, keepdims=True) + eps)
    return c * r, r


def _norm_grad(g, vh, r, kind):
    out = g - vh * (g * vh).mean(axis=1, keepdims=True)
    if kind == "layer":
        out = out - g.mean(axis=1, keepdims=True)
    return r * out


def _rows(shape, mod_id):
    B, N, _ = shape
    ids = np.repeat(np.arange(B), N) if mod_id is None else np.asarray(mod_id).reshape(-1)
    live = np.flatnonzero(ids >= 0)
    return live, ids[live]


def residual_fwd(x, h=None, gate=None, shift=None, scale=None, mod_id=None, weight=None, bias=None, post_weight=None,
                 norm="layer", post_norm=None, alpha=1.0, eps=1e-6):
    """(x_out, y, xh, factor): xh the normalised x_out and factor = weight (1 + scale), both 0 on padding."""
    shape = x.shape
    D = shape[2]
    live, s = _rows(shape, mod_id)
    x = _f64(x).reshape(-1, D)
    t = x.copy()
    if h is not None:
        u = _f64(h).reshape(-1, D)[live]
        if post_norm:
            u = _norm(u, post_norm, eps)[0]
        if post_weight is not None:
            u = u * _f64(post_weight)
        if gate is not None:
            u = u * _f64(gate)[s]
        t[live] = alpha * x[live] + u
    xh = np.zeros_like(t)
    factor = np.zeros_like(t)
    y = np.zeros_like(t)
    xh[live] = _norm(t[live], norm, eps)[0]
    factor[live] = 1.0 if scale is None else 1.0 + _f64(scale)[s]
    n = xh[live] if weight is None else xh[live] * _f64(weight)
    n = n if bias is None else n + _f64(bias)
    y[live] = n * factor[live] + (0.0 if shift is None else _f64(shift)[s])
    if weight is not None:
        factor = factor * _f64(weight)
    return t.reshape(shape), y.reshape(shape), xh.reshape(shape), factor.reshape(shape)


def residual_bwd(dx_out, dy, x_out, h=None, gate=None, shift=None, scale=None, mod_id=None, weight=None, bias=None,
                 post_weight=None, norm="layer", post_norm=None, alpha=1.0, eps=1e-6):
    """Gradients by name, and under name + "_mag" the sum of the magnitudes a summed gradient adds."""
    shape = x_out.shape
    D = shape[2]
    live, s = _rows(shape, mod_id)
    gate, scale, weight, bias, post_weight = map(_opt, (gate, scale, weight, bias, post_weight))
    full = np.zeros((shape[0] * shape[1], D)) if dx_out is None else _f64(dx_out).reshape(-1, D).copy()
    dy = _f64(dy).reshape(-1, D)[live]
    xh, r = _norm(_f64(x_out).reshape(-1, D)[live], norm, eps)
    one = 1.0 if scale is None else 1.0 + scale[s]
    w = 1.0 if weight is None else weight
    out = {}

    def by_row(name, table, terms):
        if table is None:
            return
        for suffix, v in (("", terms), ("_mag", np.abs(terms))):
            acc = np.zeros(table.shape)
            np.add.at(acc, s, v)
            out[name + suffix] = acc

    def over_rows(name, vector, terms):
        if vector is not None:
            out[name], out[name + "_mag"] = terms.sum(axis=0), np.abs(terms).sum(axis=0)

    by_row("dshift", _opt(shift), dy)
    by_row("dscale", scale, dy * (xh * w + (0.0 if bias is None else bias)))
    over_rows("dweight", weight, dy * one * xh)
    over_rows("dbias", bias, dy * one)
    t = full[live] + _norm_grad(dy * one * w, xh, r, norm)
    full[live] = alpha * t
    out["dx"] = full.reshape(shape)
    if h is not None or post_norm is None:
        hh = np.zeros_like(t) if h is None else _f64(h).reshape(-1, D)[live]
        rh = None
        if post_norm:
            hh, rh = _norm(hh, post_norm, eps)
        w2 = 1.0 if post_weight is None else post_weight
        by_row("dgate", gate, t * hh * w2)
        g = 1.0 if gate is None else gate[s]
        over_rows("dpost_weight", post_weight, t * g * hh)
        dz = t * g * w2
        dh = np.zeros_like(full)
        dh[live] = dz if rh is None else _norm_grad(dz, hh, rh, post_norm)
        out["dh"] = dh.reshape(shape)
    return out
