"""The oracle of positions, rotary positions and the gated residual: closed
forms, torch fp64 autograd and finite differences (CPU only)."""

import math

import numpy as np
import pytest
import torch

import oracle


def test_positions_restart_in_each_segment():
    p = oracle.positions([[2, 0, 3], [1, 1, 1]], 4, 22, axes=1)[..., 0]
    assert p[0].tolist() == list(range(8)) + list(range(12)) + [0, 0]
    assert p[1].tolist() == list(range(4)) * 3 + [0] * 10
    q = oracle.positions([[2, 0, 3], [1, 1, 1]], 4, 22, axes=3, row_width=3)
    assert q[0, 8 + 7].tolist() == [1, 1, 0] and q[0, 8 + 6].tolist() == [1, 0, 2]


def test_angles_of_far_positions_are_exact():
    """cos(2^31 radians) and others, against mpmath-free identities: angle doubling from a near position."""
    f = 0.7371
    far = oracle.rotary_angles(np.full((1, 1, 1), 1 << 20), [f], (1,))[0, 0, 0]
    c, s = math.cos(f), math.sin(f)          # exact fraction of the same double
    z = complex(c, s)
    for _ in range(20):                      # 2^20 by squaring; each squaring doubles the error
        z = z * z
    assert abs(z - complex(math.cos(far), math.sin(far))) < (1 << 20) * 4e-16
    neg = oracle.rotary_angles(np.full((1, 1, 1), -5), [f], (1,))[0, 0, 0]
    assert abs(math.cos(neg) - math.cos(5 * f)) < 1e-14 and abs(math.sin(neg) + math.sin(5 * f)) < 1e-14


@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_dot_products_depend_on_the_distance_only(layout):
    rng = np.random.default_rng(0)
    x, y = rng.standard_normal((2, 1, 1, 1, 16))
    f = 10000.0 ** (-np.arange(8) / 8)

    def dot(i, j):
        p = [np.full((1, 1, 1), v) for v in (i, j)]
        return float((oracle.rotary_fwd(x, p[0], f, (8,), layout) * oracle.rotary_fwd(y, p[1], f, (8,), layout)).sum())

    assert abs(dot(3, 11) - dot(100003, 100011)) < 1e-11
    assert abs(dot(0, 0) - float((x * y).sum())) < 1e-13


@pytest.mark.parametrize("norm", [None, "head", "token"])
@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_rotary_gradient_against_differences(norm, layout):
    rng = np.random.default_rng(1)
    B, L, H, D, R = 1, 2, 2, 6, 4
    x, dout = rng.standard_normal((2, B, L, H, D))
    w = None if norm is None else rng.standard_normal(H * D if norm == "token" else D)
    pos = rng.integers(-50, 50, (B, L, 2))
    f = np.array([1.0, 0.3])
    kw = dict(sections=(1, 1), layout=layout, gain=1.3, norm=norm, eps=1e-3)

    def val(x, w):
        return float((oracle.rotary_fwd(x, pos, f, weight=w, **kw) * dout).sum())

    dx, dw, _ = oracle.rotary_bwd(dout, pos, f, x=x, weight=w, **kw)
    e = 1e-6
    for i in np.ndindex(x.shape):
        d = np.zeros_like(x)
        d[i] = e
        assert abs((val(x + d, w) - val(x - d, w)) / (2 * e) - dx[i]) < 1e-7
    for i in range(0 if w is None else w.size):
        d = np.zeros_like(w)
        d[i] = e
        assert abs((val(x, w + d) - val(x, w - d)) / (2 * e) - dw[i]) < 1e-7


@pytest.mark.parametrize("norm,post,full", [("layer", None, True), ("rms", "rms", True), ("layer", "layer", True),
                                            ("rms", None, False)])
def test_residual_against_autograd(norm, post, full):
    g = torch.Generator().manual_seed(2)
    B, N, D, S = 2, 5, 8, 3
    r = lambda *s: torch.randn(*s, generator=g, dtype=torch.float64)  # noqa: E731
    x, h, dxo, dy = (r(B, N, D) for _ in range(4))
    gate, shift, scale = (r(S, D) for _ in range(3)) if full else (None,) * 3
    w = r(D) if full else None
    b = r(D) if full and norm == "layer" else None
    w2 = r(D) if post else None
    ids = torch.tensor([[0, 0, 1, -1, -1], [1, 2, 2, 2, -1]])
    live = (ids >= 0)[..., None]
    s = ids.clamp(min=0)

    def nrm(v, kind):
        v = v - v.mean(2, keepdim=True) if kind == "layer" else v
        return v / (v.pow(2).mean(2, keepdim=True) + 1e-3).sqrt()

    def branch(h, gate, w2):
        u = nrm(h, post) if post else h
        u = u if w2 is None else u * w2
        return u if gate is None else u * gate[s]

    def outer(t, w, b, scale, shift):
        n = nrm(t, norm)
        n = n if w is None else n * w
        n = n if b is None else n + b
        n = n if scale is None else n * (1 + scale[s])
        n = n if shift is None else n + shift[s]
        return torch.where(live, n, torch.zeros_like(n))

    args = [gate, shift, scale]
    kw = dict(mod_id=ids.numpy(), weight=w, bias=b, post_weight=w2, norm=norm, post_norm=post, alpha=0.6, eps=1e-3)
    t, y, _, _ = oracle.residual_fwd(x, h, *args, **kw)
    T = torch.where(live, 0.6 * x + branch(h, gate, w2), x)
    np.testing.assert_allclose(t, T, atol=1e-13)
    np.testing.assert_allclose(y, outer(T, w, b, scale, shift), atol=1e-12)
    got = oracle.residual_bwd(dxo, dy, T, h, *args, **kw)
    lf = {k: v.clone().requires_grad_() for k, v in dict(t=T, h=h, gate=gate, shift=shift, scale=scale, w=w, b=b,
                                                         w2=w2).items() if v is not None}
    (outer(lf["t"], lf.get("w"), lf.get("b"), lf.get("scale"), lf.get("shift")) * dy).sum().backward()
    dt = dxo + lf["t"].grad
    np.testing.assert_allclose(got["dx"], torch.where(live, 0.6 * dt, dxo), atol=1e-12)
    (branch(lf["h"], lf.get("gate"), lf.get("w2")) * torch.where(live, dt, torch.zeros_like(dt))).sum().backward()
    for mine, theirs in (("dh", "h"), ("dgate", "gate"), ("dshift", "shift"), ("dscale", "scale"), ("dweight", "w"),
                         ("dbias", "b"), ("dpost_weight", "w2")):
        if theirs in lf:
            np.testing.assert_allclose(got[mine], lf[theirs].grad, atol=1e-11)
        else:
            assert mine not in got
