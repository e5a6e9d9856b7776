"""pack_build_positions, pack_rotary_fwd / _bwd against the fp64 oracle (GPU).

Tolerances, from the arithmetic.  A bf16 result is off by at most half a step,
2^-8 of its value.  Before that rounding: the angle is exact to 2^-32 turns and
is rounded once to fp32 (at most pi 2^-24), sin and cos on [-pi, pi] are off by
at most 2^-20.9, so a turned feature is off by at most 2^-19 of its pair's
magnitude; a norm adds the error of its sum (a chain of at most 64 fp32
additions for up to 12,288 features, 2^-18, halved by the root) and of rsqrt
and the products (2^-21).  Together below 2^-15 of the pair's magnitude
forward.  Backward the norm's gradient subtracts two terms: the bound is taken
on r (|g w| + |xh| |mean|), at most 2^-14 of it.  A weight gradient adds terms
that are off by 2^-15 of a magnitude the pair shares, in fp32 chains below
2^8 long (2^-16): at most 2^-13 of the sum of magnitudes over the pair.
"""

import math

import numpy as np
import pytest
import torch

import oracle

pytestmark = pytest.mark.gpu
STEP = torch.finfo(torch.bfloat16).eps / 2


@pytest.fixture(scope="module")
def pvl(cuda_ok):
    import packed_variable_length_gb300 as p
    return p


def f64(t):
    return t.detach().to("cpu", torch.float64).numpy()


def pair_magnitude(v, R, layout):
    """Each feature's pair magnitude (the feature's own past R)."""
    out = np.abs(v)
    first, second = (slice(0, R // 2), slice(R // 2, R)) if layout == "half" else (slice(0, R, 2), slice(1, R, 2))
    m = np.hypot(v[..., first], v[..., second])
    out[..., first] = m
    out[..., second] = m
    return out


def near(name, got, ref, mag):
    assert np.isfinite(got).all(), name
    err = np.abs(got - ref) - STEP * np.abs(ref) - mag
    assert err.max() <= 0, f"{name}: {np.count_nonzero(err > 0)} values out of tolerance, worst by {err.max():.3e}"


def freqs_of(sections, base=10000.0):
    return np.concatenate([base ** (-np.arange(n) / n) for n in sections])


def make(B, L, H, Hk, D, R, axes, layout, norm, seed, far=0, fused=False, weights=True):
    g = torch.Generator().manual_seed(seed)
    rnd = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    if fused:
        qkv = rnd(B, L, H + 2 * Hk, D).to(torch.bfloat16).cuda()
        q, k = qkv[:, :, :H], qkv[:, :, H:H + Hk]
    else:
        q, k = rnd(B, L, H, D).to(torch.bfloat16).cuda(), rnd(B, L, Hk, D).to(torch.bfloat16).cuda()
    dq, dk = rnd(B, L, H, D).to(torch.bfloat16).cuda(), rnd(B, L, Hk, D).to(torch.bfloat16).cuda()
    wq = wk = None
    if norm and weights:
        wq = (1 + 0.2 * rnd(H * D if norm == "token" else D)).cuda()
        wk = (1 + 0.2 * rnd(Hk * D if norm == "token" else D)).cuda()
    pos = torch.randint(-100, 400, (B, L, axes), generator=g, dtype=torch.int64) + far
    n = R // 2 // axes
    sections = (R // 2 - n * (axes - 1),) + (n,) * (axes - 1)
    return q, k, dq, dk, wq, wk, pos.clamp(-2 ** 31, 2 ** 31 - 1).to(torch.int32).cuda(), sections


def check(pvl, case, seed=0, **extra):
    B, L, H, Hk, D, R, axes, layout, norm = case
    q, k, dq, dk, wq, wk, pos, sections = make(*case, seed, **extra)
    plan = pvl.rotary_plan(R, layout=layout, sections=sections, gain=1.25)
    qo, ko = pvl.pack_rotary_fwd(q, k, pos, plan, norm, wq, wk, eps=1e-5)
    gq, gk, gwq, gwk = pvl.pack_rotary_bwd(dq, dk, pos, plan, norm, q, k, wq, wk, eps=1e-5)
    pvl.device_error()
    kw = dict(pos=pos.cpu().numpy(), freqs=freqs_of(sections), sections=sections, layout=layout, gain=1.25, norm=norm,
              eps=1e-5)
    for name, x, out, dout, gx, w, gw in (("q", q, qo, dq, gq, wq, gwq), ("k", k, ko, dk, gk, wk, gwk)):
        ref = oracle.rotary_fwd(x, weight=w, **kw)
        near(name, f64(out), ref, 2.0 ** -15 * pair_magnitude(ref, R, layout))
        rdx, rdw, mag = oracle.rotary_bwd(dout, x=x, weight=w, **kw)
        g0 = pair_magnitude(oracle.rotary_bwd(dout, **{**kw, "norm": None})[0], R, layout)
        if norm is None:
            near("d" + name, f64(gx), rdx, 2.0 ** -15 * g0)
            assert gw is None
            continue
        xs = f64(x)
        r, ax = oracle.rotary._rms(xs, norm, 1e-5)
        ww = np.abs(oracle.rotary._weight(w, xs, norm))
        amag = r * (g0 * ww + np.abs(xs * r) * (g0 * ww * np.abs(xs * r)).mean(axis=ax, keepdims=True))
        near("d" + name, f64(gx), rdx, 2.0 ** -14 * amag)
        if w is None:
            assert gw is None
            continue
        over = (0, 1) if norm == "token" else (0, 1, 2)
        near("dw" + name, f64(gw), rdw, 2.0 ** -13 * (g0 * np.abs(xs * r)).sum(axis=over).ravel())


@pytest.mark.parametrize("axes,row", [(1, None), (2, None), (3, 6)])
def test_positions(pvl, axes, row):
    rng = np.random.default_rng(axes)
    for B, K, T, L in ((1, 1, 1, 1), (2, 3, 38, 1000), (3, 7, 5, 257), (64, 32, 3, 512)):
        cuts = np.sort(rng.integers(0, L // T + 1, (B, K)), axis=1)
        frames = np.diff(cuts, axis=1, prepend=0)
        got = pvl.pack_build_positions(frames, T, L, axes=axes, row_width=row)
        np.testing.assert_array_equal(got.cpu().numpy(), oracle.positions(frames, T, L, axes, row))


@pytest.mark.parametrize("norm", [None, "head", "token"])
@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("dims", [(1, 1, 1, 1, 2, 2, 1), (2, 37, 12, 12, 128, 128, 3), (1, 70, 5, 2, 80, 80, 2),
                                  (3, 41, 16, 4, 96, 64, 1), (2, 33, 3, 1, 72, 40, 1), (1, 19, 7, 7, 54, 30, 2),
                                  (1, 9, 2, 1, 256, 250, 3), (1, 350, 1, 1, 64, 64, 1)])
def test_against_oracle(pvl, dims, layout, norm):
    check(pvl, (*dims, layout, norm))


@pytest.mark.parametrize("norm", ["head", "token"])
def test_wide_tokens(pvl, norm):
    """40 + 40 heads of 128, 12,288 features, more than one round of a team for the norm per head, and scalar loads."""
    check(pvl, (1, 21, 40, 40, 128, 128, 1, "half", norm))
    check(pvl, (1, 400, 48, 48, 128, 126, 1, "interleaved", norm))
    check(pvl, (1, 5, 200, 100, 34, 34, 1, "half", norm))


@pytest.mark.parametrize("far", [-2 ** 31 + 100, 1 << 20, 1_000_000_007, 2 ** 31 - 400])
def test_far_positions(pvl, far):
    check(pvl, (2, 40, 2, 2, 64, 64, 1, "half", None), far=far)


@pytest.mark.parametrize("norm", [None, "head", "token"])
def test_slices_of_a_projection(pvl, norm):
    check(pvl, (2, 45, 6, 3, 128, 128, 1, "interleaved", norm), fused=True)
    check(pvl, (2, 45, 6, 3, 128, 128, 1, "interleaved", norm), fused=True, weights=False)


def test_odd_strides_and_offsets(pvl):
    """Views that allow no vectors give what contiguous copies give, bit for bit where the sums' order is the same."""
    q, k, _, _, _, _, pos, sections = make(2, 30, 4, 4, 64, 64, 1, "half", None, 3)
    plan = pvl.rotary_plan(64)
    a, b = pvl.pack_rotary_fwd(q, k, pos, plan)
    buf = torch.zeros(2, 30, 4, 65, dtype=torch.bfloat16, device="cuda")
    odd = buf[..., 1:]
    odd.copy_(q)
    c, _ = pvl.pack_rotary_fwd(odd, None, pos, plan)
    assert torch.equal(a, c)
    heads_first = k.transpose(1, 2).contiguous().transpose(1, 2)
    _, d = pvl.pack_rotary_fwd(q, heads_first, pos, plan)
    assert torch.equal(b, d)
    out = torch.full((2, 30, 4, 65), 7.0, dtype=torch.bfloat16, device="cuda")
    pvl.pack_rotary_fwd(q, None, pos, plan, q_out=out[..., 1:])
    assert torch.equal(out[..., 1:], a) and bool((out[..., 0] == 7.0).all())


@pytest.mark.parametrize("norm", [None, "head", "token"])
def test_in_place(pvl, norm):
    q, k, dq, dk, wq, wk, pos, sections = make(2, 50, 6, 2, 128, 96, 1, "half", norm, 4, fused=True)
    plan = pvl.rotary_plan(96)
    a, b = pvl.pack_rotary_fwd(q, k, pos, plan, norm, wq, wk)
    ga = pvl.pack_rotary_bwd(dq, dk, pos, plan, norm, q, k, wq, wk)
    dq2, dk2 = dq.clone(), dk.clone()
    gb = pvl.pack_rotary_bwd(dq2, dk2, pos, plan, norm, q, k, wq, wk, dq=dq2, dk=dk2)
    for u, v in zip(ga, gb):
        assert (u is None and v is None) or torch.equal(u, v)
    assert gb[0] is dq2
    pvl.pack_rotary_fwd(q, k, pos, plan, norm, wq, wk, q_out=q, k_out=k)
    assert torch.equal(a, q) and torch.equal(b, k)


def test_a_row_of_zeros_and_of_nan_stays_alone(pvl):
    q, k, dq, dk, wq, wk, pos, _ = make(1, 40, 4, 4, 64, 64, 1, "half", "token", 5)
    plan = pvl.rotary_plan(64)
    a, _ = pvl.pack_rotary_fwd(q, k, pos, plan, "token", wq, wk)
    q2 = q.clone()
    q2[0, 7] = float("nan")
    q2[0, 8] = 0.0
    b, kb = pvl.pack_rotary_fwd(q2, k, pos, plan, "token", wq, wk)
    assert bool(b[0, 7].isnan().all()) and bool((b[0, 8] == 0).all()) and bool(kb.isfinite().all())
    keep = [i for i in range(40) if i not in (7, 8)]
    assert torch.equal(a[0, keep], b[0, keep])


def test_repeatable(pvl):
    q, k, dq, dk, wq, wk, pos, sections = make(2, 3000, 12, 12, 128, 128, 1, "half", "token", 6)
    plan = pvl.rotary_plan(128)
    runs = [pvl.pack_rotary_bwd(dq, dk, pos, plan, "token", q, k, wq, wk) for _ in range(2)]
    for u, v in zip(*runs):
        assert torch.equal(u, v)


def test_side_stream_and_graph(pvl):
    """Calls on two streams at once, and a captured pair replayed on new inputs."""
    q, k, dq, dk, wq, wk, pos, _ = make(2, 2000, 12, 12, 128, 128, 1, "half", "head", 7)
    plan = pvl.rotary_plan(128)

    def both(stream=None):
        return (*pvl.pack_rotary_fwd(q, k, pos, plan, "head", wq, wk, stream=stream),
                *pvl.pack_rotary_bwd(dq, dk, pos, plan, "head", q, k, wq, wk, stream=stream))

    ref = both()
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs = [both(s) for s in streams for _ in range(3)]
    torch.cuda.synchronize()
    for out in outs:
        for u, v in zip(ref, out):
            assert torch.equal(u, v)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = both()
    q.copy_(q.flip(1))
    dq.copy_(dq.flip(1))
    graph.replay()
    torch.cuda.synchronize()
    for u, v in zip(out, both()):
        assert torch.equal(u, v)


def test_plan_scalings(pvl):
    """Frequencies against their formulas in double, and the gain.  The table is a fixed-point number of turns: half
    a step of 2^-64 turns is pi 2^-64 radians absolute, 2^-33 of a turn over 2^31 positions; the rest is the
    double formulas' own rounding (relative 2^-48)."""
    n, length, s = 32, 4096, 8.0
    half = math.pi * 2.0 ** -64

    def radians(**kw):
        return pvl.rotary_plan(2 * n, device="cpu", **kw).turns.numpy().astype(np.float64) / 2.0 ** 64 * 2 * math.pi

    f = 10000.0 ** (-np.arange(n) / n)
    np.testing.assert_allclose(radians(), f, rtol=2.0 ** -48, atol=half)
    np.testing.assert_allclose(radians(scaling="linear", factor=s), f / s, rtol=2.0 ** -48, atol=half)
    got = radians(scaling="ntk", factor=s)
    np.testing.assert_allclose(got[[0, -1]], [1.0, f[-1] / s], rtol=2.0 ** -44, atol=half)
    got = radians(scaling="parts", factor=s, length=length)
    turns = length * f / (2 * math.pi)
    np.testing.assert_allclose(got[turns >= 32], f[turns >= 32], rtol=2.0 ** -48, atol=half)
    np.testing.assert_allclose(got[turns <= 1], f[turns <= 1] / s, rtol=2.0 ** -48, atol=half)
    assert ((got < f) & (got > f / s))[(turns < 32) & (turns > 1)].all()
    assert pvl.rotary_plan(8, scaling="parts", factor=s, length=9, device="cpu").gain == 0.1 * math.log(s) + 1


def test_refusals(pvl):
    q, k, dq, dk, wq, wk, pos, _ = make(2, 10, 4, 4, 64, 64, 1, "half", "token", 8)
    plan = pvl.rotary_plan(64)
    bad = [dict(q=q.float()), dict(q=q[..., ::2]), dict(k=k[:1]), dict(positions=pos.long()), dict(positions=pos[:, :5]),
           dict(norm="rms"), dict(norm="head"), dict(norm=None), dict(q_weight=wq[:64].contiguous()),
           dict(q_weight=wq.double()), dict(k=None), dict(q=q.cpu()), dict(q_out=torch.empty_like(q)[:, :9])]
    for change in bad:
        kw = {**dict(q=q, k=k, positions=pos, plan=plan, norm="token", q_weight=wq, k_weight=wk), **change}
        with pytest.raises(ValueError):
            pvl.pack_rotary_fwd(**kw)
    with pytest.raises(ValueError):
        pvl.pack_rotary_bwd(dq, dk, pos, plan, "token", None, None, wq, wk)
    with pytest.raises(pvl.PvlError):
        pvl.pack_rotary_fwd(q, k, pos, pvl.rotary_plan(66))           # more than the head
    with pytest.raises(pvl.PvlError):
        big = torch.empty(1, 2, 1, 258, dtype=torch.bfloat16, device="cuda")
        pvl.pack_rotary_fwd(big, None, pos[:1, :2].contiguous(), plan)
    with pytest.raises(pvl.PvlError):                                 # a token that no block holds
        wide = torch.empty(1, 2, 600, 66, dtype=torch.bfloat16, device="cuda")
        pvl.pack_rotary_fwd(wide, None, pos[:1, :2].contiguous(), plan, "token")
    with pytest.raises(pvl.PvlError):
        pvl.pack_rotary_fwd(q, k, pos, plan, "token", wq, wk, eps=-1.0)


@pytest.mark.parametrize("norm", [None, "head", "token"])
def test_autograd(pvl, norm):
    """The wrapper's gradients are the backward call's, with shared leaves and with an output left out."""
    q, k, dq, dk, wq, wk, pos, sections = make(2, 26, 6, 3, 64, 48, 1, "half", norm, 9)
    plan = pvl.rotary_plan(48)
    leaves = [t.clone().requires_grad_() if t is not None else None for t in (q, k, wq, wk)]
    qo, ko = pvl.packed_rotary(leaves[0], leaves[1], pos, plan, norm, leaves[2], leaves[3])
    grads = torch.autograd.grad([qo, ko], [t for t in leaves if t is not None], [dq, dk])
    ref = [t for t in pvl.pack_rotary_bwd(dq, dk, pos, plan, norm, q, k, wq, wk) if t is not None]
    for u, v in zip(grads, ref):
        assert torch.equal(u, v)
    only = pvl.packed_rotary(leaves[0], None, pos, plan, norm, leaves[2])
    assert torch.equal(only, qo)
    qo, ko = pvl.packed_rotary(leaves[0], leaves[1], pos, plan, norm, leaves[2], leaves[3])
    g = torch.autograd.grad(qo.float().sum(), leaves[0])[0]           # expanded ones come back
    assert torch.equal(g, pvl.pack_rotary_bwd(torch.ones_like(dq), torch.zeros_like(dk), pos, plan, norm, q, k, wq,
                                              wk)[0])


def test_offsets_past_32_bits(pvl):
    """A projection of 2.4 G elements: the last tokens are what the same call gives on a copy of them."""
    L, H, D = 524289, 12, 128
    qkv = torch.empty(1, L, 3 * H, D, dtype=torch.bfloat16, device="cuda")
    tail = torch.randn(1, 77, 3 * H, D, device="cuda").to(torch.bfloat16)
    qkv[:, :-77] = 1.0
    qkv[:, -77:] = tail
    pos = torch.arange(L, dtype=torch.int32, device="cuda")[None]
    plan = pvl.rotary_plan(D)
    for norm in (None, "token"):
        a, b = pvl.pack_rotary_fwd(qkv[:, :, H:2 * H], qkv[:, :, 2 * H:], pos, plan, norm)
        c, d = pvl.pack_rotary_fwd(tail[:, :, H:2 * H], tail[:, :, 2 * H:], pos[:, -77:].contiguous(), plan, norm)
        # one team a token either way, but other lanes may add its squares: half a step apart at most
        assert torch.equal(a[:, -77:], c) if norm is None else bool(((a[:, -77:] - c).abs() <= 2.0 ** -7 * c.abs()).all())
        assert torch.equal(b[:, -77:], d) if norm is None else bool(((b[:, -77:] - d).abs() <= 2.0 ** -7 * d.abs()).all())
        del a, b
    pvl.device_error()


def test_one_token_of_many_rows(pvl):
    """Serving: one token of each of 70,000 sequences, heads first in memory."""
    B, H, D = 70000, 2, 32
    q = torch.randn(B, H, 1, D, device="cuda").to(torch.bfloat16).transpose(1, 2)
    k = torch.randn(B, 1, 1, D, device="cuda").to(torch.bfloat16)
    pos = torch.randint(0, 1 << 20, (B, 1), dtype=torch.int32, device="cuda")
    plan = pvl.rotary_plan(D)
    a, b = pvl.pack_rotary_fwd(q, k, pos, plan, "head")
    c, d = pvl.pack_rotary_fwd(q.transpose(0, 1).contiguous(), k.transpose(0, 1).contiguous(), pos.t().contiguous(), plan,
                               "head")
    assert torch.equal(a.transpose(0, 1), c) and torch.equal(b.transpose(0, 1), d)
