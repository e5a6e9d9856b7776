"""Oracle: log-probabilities of tokens, the preference loss over pairs of
packed episodes and the clipped policy loss, with their gradients, fp64 on the
CPU.  TEST INFRASTRUCTURE ONLY (see the package docstring).

Tokens carry episode ids as in attention: a negative id takes no part.
"""

from __future__ import annotations

import math

import numpy as np

from .loss import _f64


def valid_targets(targets, V: int, seq_id=None) -> np.ndarray:
    """[B, L]: tokens with an id whose target is one of the V."""
    t = np.asarray(targets)
    ok = (t >= 0) & (t < V)
    return ok if seq_id is None else ok & (np.asarray(seq_id) >= 0)


def logprob(logits, targets, valid, temperature: float = 1.0):
    """(logp, lse, entropy) [B, L] of targets under softmax(logits / T); zeros where not valid."""
    x, t = _f64(logits), np.asarray(targets)
    out = np.zeros((3,) + t.shape)
    for at in np.argwhere(valid):
        at = tuple(at)
        top = x[at].max()
        d = (x[at] - top) / temperature     # before the sum's logarithm, which a large top would absorb
        e = np.exp(d)
        logs = math.log(e.sum())
        p = e / e.sum()
        out[0][at] = d[t[at]] - logs
        out[1][at] = top / temperature + logs
        out[2][at] = -np.sum(p[p > 0] * (d[p > 0] - logs))
    return out[0], out[1], out[2]


def logprob_grad(logits, targets, valid, dlogp=None, dentropy=None, temperature: float = 1.0):
    """Gradient [B, L, V] to the logits."""
    x, t = _f64(logits), np.asarray(targets)
    g = np.zeros_like(x)
    _, _, ent = logprob(logits, targets, valid, temperature)
    for at in np.argwhere(valid):
        at = tuple(at)
        z = (x[at] - x[at].max()) / temperature
        z = z - math.log(np.exp(z).sum())
        p = np.exp(z)
        if dlogp is not None:
            up = float(_f64(dlogp)[at])
            g[at] -= up * p
            g[at][t[at]] += up
        if dentropy is not None:
            g[at] -= float(_f64(dentropy)[at]) * p * np.where(p > 0, z + ent[at], 0.0)
        g[at] /= temperature
    return g


def _sums(v, ids, E: int):
    """(sum over each episode's tokens, their number)."""
    ids = np.asarray(ids).reshape(-1)
    ok = ids >= 0
    s, n = np.zeros(E), np.zeros(E)
    np.add.at(s, ids[ok], np.asarray(v, dtype=np.float64).reshape(-1)[ok])
    np.add.at(n, ids[ok], 1.0)
    return s, n


def _spread(table, ids):
    ids = np.asarray(ids)
    return np.where(ids >= 0, np.asarray(table)[np.maximum(ids, 0)], 0.0)


def preference(logp, ref_logp, seq_id, pairs, E: int, beta=0.1, kind="sigmoid", smoothing=0.0, margin=0.0, mean=False):
    """(loss, rewards [P, 2], coef [E], dlogp like seq_id)."""
    lp = _f64(logp)
    d = lp - (0.0 if ref_logp is None else _f64(ref_logp))
    D, n = _sums(np.where(np.asarray(seq_id) >= 0, d, 0.0), seq_id, E)
    each = 1.0 / np.maximum(n, 1.0) if mean else np.ones(E)
    D = D * each
    pairs = np.asarray(pairs)
    rewards, up, loss, count = np.zeros(pairs.shape), np.zeros(E), 0.0, 0
    for i, (c, r) in enumerate(pairs):
        if c < 0 or r < 0:
            continue
        count += 1
        rewards[i] = beta * D[c], beta * D[r]
        h = D[c] - D[r] - margin
        x = beta * h
        if kind == "sigmoid":
            loss += (1 - smoothing) * np.logaddexp(0.0, -x) + smoothing * np.logaddexp(0.0, x)
            g = beta * (smoothing - math.exp(-np.logaddexp(0.0, x)))
        elif kind == "squared":
            loss += (h - 0.5 / beta) ** 2
            g = 2.0 * (h - 0.5 / beta)
        else:
            loss += max(0.0, 1.0 - x)
            g = -beta if x < 1.0 else 0.0
        up[c] += g
        up[r] -= g
    coef = up * each / max(count, 1)
    return loss / max(count, 1), rewards, coef, _spread(coef, seq_id)


def policy(logp, old_logp, advantages, seq_id, E: int, ref_logp=None, clip_low=0.2, clip_high=0.2, kl_weight=0.0,
           ratio="token", mean="token"):
    """(loss, divergence, share of clipped ratios, dlogp like seq_id)."""
    ids = np.asarray(seq_id)
    ok = ids >= 0
    lp = _f64(logp)
    d = np.zeros(ids.shape) if old_logp is None else np.where(ok, lp - _f64(old_logp), 0.0)
    _, n = _sums(d, ids, E)
    tokens, some = n.sum(), (n > 0).sum()
    weight = np.ones(E) / max(tokens, 1) if mean == "token" else 1.0 / (np.maximum(n, 1) * max(some, 1))
    w = _spread(weight, ids)
    A = _f64(advantages)
    per_token = ratio == "token" and A.shape == ids.shape
    if ratio == "episode":
        d = _spread(_sums(d, ids, E)[0] / np.maximum(n, 1), ids)
    a = A if per_token else _spread(A, ids)
    a = np.where(ok, a, 0.0)
    cut = np.where(a > 0, d > math.log1p(clip_high), (a < 0) & (d < math.log1p(-clip_low)))
    r = np.exp(np.where(cut | (a == 0), 0.0, d))
    r = np.where(cut, np.where(a > 0, 1.0 + clip_high, 1.0 - clip_low), r)
    loss = -(w * r * a).sum()
    grad = np.where(cut, 0.0, -w * r * a)
    kl = 0.0
    if ref_logp is not None:
        f = np.where(ok, _f64(ref_logp) - np.where(ok, lp, 0.0), 0.0)
        kl = (w * (np.expm1(f) - f)).sum()
        loss += kl_weight * kl
        grad = grad - kl_weight * w * np.expm1(f)
    if ratio == "episode":
        share = len(np.unique(ids[cut & ok])) / max(some, 1)
    else:
        share = (cut & ok).sum() / max(tokens, 1)
    return loss, kl, share, grad
