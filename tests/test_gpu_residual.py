"""adaln_residual_fwd / _bwd against the fp64 oracle (GPU), and the run of
positions, rotary, attention and the gated residual together.

Tolerances, from the arithmetic.  A bf16 result is off by at most half a step
(2^-8 of its value), an fp32 one by 2^-24.  Before that rounding the kernels
work in fp32.  A row's sums are chains of at most 64 additions (2^-18 of the
sum of magnitudes); they are shifted by the row's first element K, and with
(mean - K)^2 at most 15 variances (so for the inputs here: K is drawn from the
row) the variance is off by at most 2^-14, the root by 2^-15, the mean by
2^-16 deviations.  So xh is off by 2^-14 (1 + |xh|), y by 2^-13 of
|factor| (1 + |xh|) + |shift| + |bias factor|, a plain x_out by 2^-22 of its
terms and one with a post norm by 2^-13 of them.  dx and dh subtract means of
products of such values: 2^-12 of r (|g| + mean |g| + |xh| mean |g xh|) + |dx_out|.
Sums over tokens add terms that are off by 2^-13 of their (1 + |xh|)-scaled
magnitudes in fp32 chains below 2^9 long: 2^-12 of the sum of magnitudes.
"""

import numpy as np
import pytest
import torch

import oracle

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def pvl(cuda_ok):
    import packed_variable_length_gb300 as p
    return p


def f64(t):
    return t.detach().to("cpu", torch.float64).numpy()


def near(name, got, ref, mag):
    """got a tensor: half a step of its type, and mag."""
    step = torch.finfo(got.dtype).eps / 2
    got = f64(got)
    assert np.isfinite(got).all(), name
    err = np.abs(got - ref) - step * np.abs(ref) - mag
    assert err.max() <= 0, f"{name}: {np.count_nonzero(err > 0)} values out of tolerance, worst by {err.max():.3e}"


def ids_of(B, N, kind, seed):
    """int32 [B, N] non-decreasing ids with padding, and the number of rows S; None for one row per batch row."""
    if kind == "batch":
        return None, B
    rng = np.random.default_rng(seed)
    run = {"episode": max(1, N // 3), "frame": 5, "token": 1}[kind]
    ids = np.empty((B, N), np.int32)
    at = 0
    for b in range(B):
        ids[b] = at + np.arange(N) // run
        at = int(ids[b].max()) + 1 + int(rng.integers(0, 2))       # some ids have no token
        if kind != "token":
            ids[b, N - int(rng.integers(0, N // 3 + 1)):] = -1
            ids[b, rng.random(N) < 0.1] = -1
    return ids, at


def make(B, N, D, kind, norm, post, stream, seed, tables=True, vectors=True):
    g = torch.Generator().manual_seed(seed)
    rnd = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    st = torch.float32 if stream == "fp32" else torch.bfloat16
    ids, S = ids_of(B, N, kind, seed)
    t = dict(x=(2 * rnd(B, N, D) + rnd(B, N, 1)).to(st).cuda(), h=rnd(B, N, D).to(torch.bfloat16).cuda(),
             dx_out=rnd(B, N, D).to(st).cuda(), dy=rnd(B, N, D).to(torch.bfloat16).cuda())
    args = [0.5 * rnd(S, D).cuda(), rnd(S, D).cuda(), 0.3 * rnd(S, D).cuda()] if tables else [None] * 3
    how = dict(mod_id=None if ids is None else torch.from_numpy(ids).cuda(),
               weight=(1 + 0.2 * rnd(D)).cuda() if vectors else None,
               bias=rnd(D).cuda() if vectors and norm == "layer" else None,
               post_weight=(1 + 0.2 * rnd(D)).cuda() if vectors and post else None, norm=norm, post_norm=post,
               alpha=0.75, eps=1e-5)
    return t, args, how


def host(how, args):
    h = {k: v.cpu() if isinstance(v, torch.Tensor) else v for k, v in how.items()}
    if h["mod_id"] is not None:
        h["mod_id"] = h["mod_id"].numpy()
    return h, [None if a is None else a.cpu() for a in args]


def check(pvl, t, args, how, branch=True):
    h = t["h"] if branch else None
    x_out, y = pvl.adaln_residual_fwd(t["x"], h, *args, **how)
    pvl.device_error()
    hh, ha = host(how, args)
    X, Y, XH, F = oracle.residual_fwd(t["x"].cpu(), None if h is None else h.cpu(), *ha, **hh)
    big = 2.0 ** -13 if how["post_norm"] else 2.0 ** -22
    terms = np.abs(f64(t["x"])) + np.abs(X) + 4.0      # |alpha x| + |gate u|, with u below 4 on average past it
    near("x_out", x_out, X, big * terms if branch else 0.0)
    shift = 0.0 if ha[1] is None else float(ha[1].abs().max())
    bias = 0.0 if hh["bias"] is None else np.abs(F).max() * float(hh["bias"].abs().max())
    near("y", y, Y, 2.0 ** -13 * (np.abs(F) * (1 + np.abs(XH)) + shift + bias))
    G = pvl.adaln_residual_bwd(t["dx_out"], t["dy"], x_out, h, *args, **how)
    pvl.device_error()
    dx_out = None if t["dx_out"] is None else t["dx_out"].cpu()
    R = oracle.residual_bwd(dx_out, t["dy"].cpu(), x_out.cpu(), None if h is None else h.cpu(), *ha, **hh)
    check_grads(G, R, t, x_out, how, ha, hh, branch)
    return x_out, y, G


def check_grads(G, R, t, x_out, how, ha, hh, branch):
    live, s = oracle.residual._rows(x_out.shape, hh["mod_id"])
    D = x_out.shape[2]
    flat = lambda v: f64(v).reshape(-1, D)  # noqa: E731
    xh, r = oracle.residual._norm(flat(x_out)[live], how["norm"], how["eps"])
    g = np.abs(flat(t["dy"])[live])
    g = g if ha[2] is None else g * np.abs(1 + f64(ha[2])[s])
    g = g if hh["weight"] is None else g * np.abs(f64(hh["weight"]))
    mean = lambda v: v.mean(axis=1, keepdims=True)  # noqa: E731
    tm = r * (g + mean(g) + np.abs(xh) * mean(g * np.abs(xh)))
    tm = tm + (0.0 if t["dx_out"] is None else np.abs(flat(t["dx_out"])[live]))
    mag = np.zeros((x_out.shape[0] * x_out.shape[1], D))
    mag[live] = tm
    near("dx", G.dx, R["dx"], 2.0 ** -12 * mag.reshape(x_out.shape))
    if not branch:
        assert G.dh is None
    else:
        z = tm if ha[0] is None else tm * np.abs(f64(ha[0])[s])
        hm = np.ones_like(z)
        if how["post_norm"]:
            z = z if hh["post_weight"] is None else z * np.abs(f64(hh["post_weight"]))
            vh, rh = oracle.residual._norm(flat(t["h"])[live], how["post_norm"], how["eps"])
            hm = np.abs(vh) + 1
            z = rh * (z + mean(z) + np.abs(vh) * mean(z * np.abs(vh)))
        elif t["h"] is not None:
            hm = np.abs(flat(t["h"])[live])
        mag[:] = 0
        mag[live] = z
        near("dh", G.dh, R["dh"], 2.0 ** -12 * mag.reshape(x_out.shape))
        if G.dgate is not None:
            gm = np.zeros(G.dgate.shape)
            w2 = 1.0 if hh["post_weight"] is None else np.abs(f64(hh["post_weight"]))
            np.add.at(gm, s, tm * hm * w2)
            near("dgate", G.dgate, R["dgate"], 2.0 ** -12 * gm)
        if G.dpost_weight is not None:
            gate = 1.0 if ha[0] is None else np.abs(f64(ha[0])[s])
            near("dpost_weight", G.dpost_weight, R["dpost_weight"], 2.0 ** -12 * (tm * hm * gate).sum(axis=0))
    dym = np.abs(flat(t["dy"])[live])
    one = 1.0 if ha[2] is None else np.abs(1 + f64(ha[2])[s])
    w = 1.0 if hh["weight"] is None else np.abs(f64(hh["weight"]))
    b = 0.0 if hh["bias"] is None else np.abs(f64(hh["bias"]))
    if G.dscale is not None:
        sm = np.zeros(G.dscale.shape)
        np.add.at(sm, s, dym * ((1 + np.abs(xh)) * w + b))
        near("dshift", G.dshift, R["dshift"], 2.0 ** -12 * R["dshift_mag"])
        near("dscale", G.dscale, R["dscale"], 2.0 ** -12 * sm)
    if G.dweight is not None:
        near("dweight", G.dweight, R["dweight"], 2.0 ** -12 * (dym * one * (1 + np.abs(xh))).sum(axis=0))
    if G.dbias is not None:
        near("dbias", G.dbias, R["dbias"], 2.0 ** -12 * R["dbias_mag"])


@pytest.mark.parametrize("stream", ["bf16", "fp32"])
@pytest.mark.parametrize("norm,post", [("layer", None), ("rms", "rms"), ("layer", "layer"), ("rms", None)])
@pytest.mark.parametrize("shape", [(2, 130, 64, "episode"), (3, 257, 1536, "frame"), (1, 1, 8, "batch"),
                                   (5, 1, 520, "batch"), (2, 97, 5120, "batch"), (1, 41, 8192, "episode"),
                                   (2, 20, 2048, "token"), (2, 3001, 256, "frame")])
def test_against_oracle(pvl, shape, norm, post, stream):
    check(pvl, *make(*shape, norm, post, stream, seed=sum(shape[:3])))


@pytest.mark.parametrize("tables,vectors", [(False, False), (True, False), (False, True)])
@pytest.mark.parametrize("kind", ["batch", "episode"])
def test_absent_factors(pvl, tables, vectors, kind):
    for norm, post in (("layer", None), ("rms", "layer")):
        t, args, how = make(2, 75, 320, kind, norm, post, "bf16", 3, tables, vectors)
        check(pvl, t, args, how)
        check(pvl, {**t, "dx_out": None}, args, how)


@pytest.mark.parametrize("only", [0, 1, 2])
def test_one_table(pvl, only):
    t, args, how = make(2, 75, 320, "episode", "layer", None, "bf16", 4)
    args = [a if i == only else None for i, a in enumerate(args)]
    x_out, y = pvl.adaln_residual_fwd(t["x"], t["h"], *args, **how)
    hh, ha = host(how, args)
    X, Y, XH, F = oracle.residual_fwd(t["x"].cpu(), t["h"].cpu(), *ha, **hh)
    near("y", y, Y, 2.0 ** -13 * (np.abs(F) * (1 + np.abs(XH)) + 8 + 8 * np.abs(F)))
    G = pvl.adaln_residual_bwd(t["dx_out"], t["dy"], x_out, t["h"], *args, **how)
    R = oracle.residual_bwd(t["dx_out"].cpu(), t["dy"].cpu(), x_out.cpu(), t["h"].cpu(), *ha, **hh)
    for name in ("dgate", "dshift", "dscale"):
        got = getattr(G, name)
        assert (got is None) == (name not in R)
        if got is not None:
            assert np.linalg.norm(f64(got) - R[name]) <= 2.0 ** -12 * np.linalg.norm(R[name + "_mag"])


@pytest.mark.parametrize("kind", ["batch", "frame"])
def test_no_branch(pvl, kind):
    """Only the modulated norm; on one modulation per batch row it is adaln_fwd's up to the order of the row's sums:
    both are within half a bf16 step and 2^-13 of the magnitudes of the exact value, so within twice that of each
    other."""
    t, args, how = make(3, 70, 1024, kind, "layer", None, "bf16", 5, vectors=False)
    how["alpha"] = 1.0
    args[0] = None
    x_out, y, G = check(pvl, t, args, how, branch=False)
    assert x_out is t["x"]
    if kind == "batch":
        _, Y, XH, F = oracle.residual_fwd(t["x"].cpu(), None, *host(how, args)[1], **host(how, args)[0])
        far = np.abs(f64(y) - f64(pvl.adaln_fwd(t["x"], args[1], args[2], 1e-5)))
        each = 2.0 ** -8 * np.abs(Y) + 2.0 ** -13 * (np.abs(F) * (1 + np.abs(XH)) + float(args[1].abs().max()))
        assert bool((far <= 2 * each).all())


def test_branch_without_h_in_the_backward(pvl):
    t, args, how = make(2, 33, 256, "episode", "rms", None, "bf16", 6)
    args[0] = None
    x_out, _ = pvl.adaln_residual_fwd(t["x"], t["h"], *args, **how)
    a = pvl.adaln_residual_bwd(t["dx_out"], t["dy"], x_out, t["h"], *args, **how)
    b = pvl.adaln_residual_bwd(t["dx_out"], t["dy"], x_out, None, *args, branch=True, **how)
    for u, v in zip(a, b):
        assert (u is None and v is None) or torch.equal(u, v)


@pytest.mark.parametrize("post", [None, "layer"])
def test_padding(pvl, post):
    """Whatever stands in padding, x_out = x, y = 0, dx = dx_out, dh = 0 there and nothing changes elsewhere; a
    batch of padding alone gives zero table gradients."""
    t, args, how = make(2, 90, 512, "frame", "layer", post, "bf16", 7)
    pad = how["mod_id"] < 0
    assert bool(pad.any()) and bool((~pad).any())

    def run():
        x_out, y = pvl.adaln_residual_fwd(t["x"], t["h"], *args, **how)
        keep = x_out.clone()
        keep[pad] = float("nan")
        return x_out, y, pvl.adaln_residual_bwd(t["dx_out"], t["dy"], keep, t["h"], *args, **how)

    x0, y0, g0 = run()
    assert torch.equal(x0[pad], t["x"][pad]) and bool((y0[pad] == 0).all())
    assert torch.equal(g0.dx[pad], t["dx_out"][pad]) and bool((g0.dh[pad] == 0).all())
    t["h"][pad] = float("nan")
    t["dy"][pad] = float("inf")
    x1, y1, g1 = run()
    assert torch.equal(x0, x1) and torch.equal(y0, y1)
    for u, v in zip(g0, g1):
        assert (u is None and v is None) or torch.equal(u, v)
    how["mod_id"].fill_(-1)
    x2, y2, g2 = run()
    assert torch.equal(x2, t["x"]) and bool((y2 == 0).all())
    for u in g2[2:]:
        assert u is None or bool((u == 0).all())


def test_id_past_the_tables_is_reported(pvl):
    t, args, how = make(1, 40, 64, "episode", "layer", None, "bf16", 8)
    S = args[0].shape[0]
    how["mod_id"][:] = 0
    how["mod_id"][0, 11] = S
    x_out, y = pvl.adaln_residual_fwd(t["x"], t["h"], *args, **how)
    st, info = pvl.device_error(raise_on_error=False)
    assert st == 1 and info[0] == 3
    assert torch.equal(x_out[0, 11], t["x"][0, 11]) and bool((y[0, 11] == 0).all())
    pvl.device_error()


def test_ids_out_of_order_are_reported(pvl):
    """Forward any order holds; backward ids that return give NaN and an error, not mixed sums."""
    t, args, how = make(1, 40, 64, "episode", "layer", None, "bf16", 9)
    ids = torch.tensor([[0, 1] * 20], dtype=torch.int32, device="cuda")
    how["mod_id"] = ids
    x_out, y = pvl.adaln_residual_fwd(t["x"], t["h"], *args, **how)
    hh, ha = host(how, args)
    X, Y, XH, F = oracle.residual_fwd(t["x"].cpu(), t["h"].cpu(), *ha, **hh)
    near("y", y, Y, 2.0 ** -13 * (np.abs(F) * (1 + np.abs(XH)) + 8 + 8 * np.abs(F)))
    pvl.device_error()
    B, N, D = 1, 5000, 64                   # more rows than CTAs: the runs of a CTA return to an id
    x = torch.randn(B, N, D, device="cuda").to(torch.bfloat16)
    how = dict(mod_id=torch.tensor([[0, 1]], dtype=torch.int32, device="cuda").repeat(1, N // 2))
    G = pvl.adaln_residual_bwd(None, x, x, x, *(a[:2].contiguous() for a in args), **how)
    st, info = pvl.device_error(raise_on_error=False)
    assert st == 1 and info[0] == 4
    assert all(bool(u.isnan().all()) for u in (G.dgate, G.dshift, G.dscale)) and bool(G.dx.isfinite().all())
    pvl.device_error()


def test_in_place_and_repeatable(pvl):
    t, args, how = make(2, 700, 1536, "frame", "layer", "rms", "fp32", 10)
    a = pvl.adaln_residual_fwd(t["x"], t["h"], *args, **how)
    G = pvl.adaln_residual_bwd(t["dx_out"], t["dy"], a[0], t["h"], *args, **how)
    H = pvl.adaln_residual_bwd(t["dx_out"], t["dy"], a[0], t["h"], *args, **how)
    for u, v in zip(G, H):
        assert (u is None and v is None) or torch.equal(u, v)
    b = pvl.adaln_residual_fwd(t["x"], t["h"], *args, x_out=t["x"], y=t["h"], **how)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1]) and b[0] is t["x"]


def test_side_streams_and_graph(pvl):
    t, args, how = make(2, 3000, 1024, "frame", "layer", "rms", "bf16", 11)

    def both(stream=None):
        x_out, y = pvl.adaln_residual_fwd(t["x"], t["h"], *args, stream=stream, **how)
        return (x_out, y, *pvl.adaln_residual_bwd(t["dx_out"], t["dy"], t["x"], t["h"], *args, stream=stream, **how))

    ref = both()
    torch.cuda.synchronize()
    outs = [both(s) for s in [torch.cuda.Stream() for _ in range(2)] for _ in range(3)]
    torch.cuda.synchronize()
    for out in outs:
        for u, v in zip(ref, out):
            assert (u is None and v is None) or torch.equal(u, v)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = both()
    t["x"].copy_(t["x"].flip(0))
    t["dy"].copy_(t["dy"].flip(1))
    graph.replay()
    torch.cuda.synchronize()
    for u, v in zip(out, both()):
        assert (u is None and v is None) or torch.equal(u, v)
    pvl.device_error()


def test_refusals(pvl):
    t, args, how = make(2, 20, 64, "episode", "layer", "rms", "bf16", 12)
    x, h = t["x"], t["h"]

    def call(x=x, h=h, gate=args[0], shift=args[1], scale=args[2], **change):
        pvl.adaln_residual_fwd(x, h, gate, shift, scale, **{**how, **change})

    for change in (dict(x=x.half()), dict(x=x[:, ::2]), dict(h=h.float()), dict(h=h[:, :5].contiguous()),
                   dict(gate=args[0].to(torch.bfloat16)), dict(gate=args[0][:1].contiguous()), dict(mod_id=None),
                   dict(mod_id=how["mod_id"].long()), dict(norm="head"), dict(post_norm="token"),
                   dict(weight=how["weight"][:32].contiguous()), dict(shift=args[1].cpu()),
                   dict(x_out=torch.empty_like(x, dtype=torch.float32))):
        with pytest.raises(ValueError):
            call(**change)
    for change in (dict(eps=-1.0), dict(alpha=float("nan")), dict(h=None), dict(post_norm=None)):
        with pytest.raises(pvl.PvlError):
            call(**change)
    with pytest.raises(pvl.PvlError):
        pvl.adaln_residual_fwd(torch.empty(1, 2, 12, device="cuda"))
    with pytest.raises(pvl.PvlError):
        pvl.adaln_residual_bwd(None, t["dy"], x, None, *args, branch=True, **how)
    with pytest.raises(pvl.PvlError):
        pvl.adaln_residual_bwd(None, t["dy"], x, h, *args, ws=torch.empty(64, dtype=torch.uint8, device="cuda"), **how)


def test_autograd(pvl):
    t, args, how = make(2, 60, 256, "episode", "layer", "rms", "fp32", 13)
    leaves = [v.clone().requires_grad_() for v in (t["x"], t["h"], *args)]
    vec = {k: how[k].clone().requires_grad_() for k in ("weight", "bias", "post_weight")}
    x_out, y = pvl.gated_residual(*leaves, **{**how, **vec})
    grads = torch.autograd.grad([x_out, y], leaves + list(vec.values()), [t["dx_out"], t["dy"]])
    ref = pvl.adaln_residual_bwd(t["dx_out"], t["dy"], x_out.detach(), t["h"], *args, **how)
    for u, v in zip(grads, ref):
        assert torch.equal(u, v)
    # only one of the outputs is used
    x_out, y = pvl.gated_residual(*leaves, **{**how, **vec})
    ref = pvl.adaln_residual_bwd(None, t["dy"], x_out.detach(), t["h"], *args, **how)
    assert torch.equal(torch.autograd.grad(y, leaves[0], t["dy"])[0], ref.dx)
    x_out, y = pvl.gated_residual(*leaves, **{**how, **vec})
    g = torch.autograd.grad(x_out.sum(), leaves[0])[0]
    live = (how["mod_id"] >= 0)[..., None]
    assert torch.equal(g, torch.where(live, 0.75, 1.0).expand_as(g))


def test_offsets_past_32_bits(pvl):
    """2.3 G elements: the last rows, and the gradients of the last modulation row, are those of the same rows alone."""
    N, D, n = 450001, 5120, 61
    x = torch.ones(1, N, D, dtype=torch.bfloat16, device="cuda")
    h = torch.ones(1, N, D, dtype=torch.bfloat16, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(15)
    x[:, -n:] = torch.randn(1, n, D, generator=g, device="cuda").to(torch.bfloat16)
    h[:, -n:] = torch.randn(1, n, D, generator=g, device="cuda").to(torch.bfloat16)
    ids = torch.zeros(1, N, dtype=torch.int32, device="cuda")
    ids[:, -n:] = 1
    tabs = [torch.randn(2, D, generator=g, device="cuda") for _ in range(3)]
    x_out, y = pvl.adaln_residual_fwd(x, h, *tabs, mod_id=ids)
    tail = [t[:, -n:].contiguous() for t in (x, h, ids)]
    a, b = pvl.adaln_residual_fwd(tail[0], tail[1], *tabs, mod_id=tail[2])
    assert torch.equal(x_out[:, -n:], a) and torch.equal(y[:, -n:], b)
    del y
    G = pvl.adaln_residual_bwd(x_out, h, x_out, h, *tabs, mod_id=ids)
    T = pvl.adaln_residual_bwd(a, tail[1], a, tail[1], *tabs, mod_id=tail[2])
    assert torch.equal(G.dx[:, -n:], T.dx) and torch.equal(G.dh[:, -n:], T.dh)
    for u, v in zip(G[2:5], T[2:5]):    # other CTAs share the rows: another order of 61 fp32 additions
        assert float((u[1] - v[1]).norm()) <= 61 * 2.0 ** -23 * float(v[1].norm()) * 8
    pvl.device_error()


def test_more_ids_than_rows_a_cta(pvl):
    """Every token its own modulation row, on a batch of many CTAs, then one row for all."""
    t, args, how = make(1, 6000, 64, "token", "layer", "rms", "bf16", 16)
    check(pvl, t, args, how)
    t, args, how = make(1, 30000, 64, "batch", "rms", None, "bf16", 17)
    check(pvl, t, args, how)


def test_block_together(pvl):
    """One attention block on a packed row, forward and backward, against the formulas in fp64: positions, rotary
    with a norm over the token, masked attention, then the gated residual and the next norm.  Its bf16
    intermediates (q, k, o and, backward, their gradients) put up to four roundings of 2^-8 in a row: 2^-5 of
    the results' norm holds them with the sums' spread."""
    frames, valid, T, L, H, D = [[3, 4], [5, 1]], [[2, 4], [5, 0]], 38, 288, 2, 64
    B, W = 2, H * D
    g = torch.Generator().manual_seed(14)
    rnd = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    x, q, k, v = (rnd(B, L, W).to(torch.bfloat16) for _ in range(4))
    gate, shift, scale = 0.5 * rnd(4, W), rnd(4, W), 0.3 * rnd(4, W)
    wq, wk = 1 + 0.2 * rnd(W), 1 + 0.2 * rnd(W)
    dx_out, dy = rnd(B, L, W).to(torch.bfloat16), rnd(B, L, W).to(torch.bfloat16)
    sections = (12, 10, 10)

    sid = pvl.pack_build_seq_ids(frames, valid, T, L)
    pos = pvl.pack_build_positions(frames, T, L, axes=3, row_width=6)
    plan = pvl.rotary_plan(D, sections=sections)
    dev = [t.cuda().requires_grad_() for t in (x, q, k, v, gate, shift, scale, wq, wk)]
    X, Q, K, V, GA, SH, SC, WQ, WK = dev
    heads = lambda t: t.view(B, L, H, D)  # noqa: E731
    qr, kr = pvl.packed_rotary(heads(Q), heads(K), pos, plan, "token", WQ, WK)
    o = pvl.packed_attention(qr, kr, heads(V), sid)
    x_out, y = pvl.gated_residual(X, o.view(B, L, W), GA, SH, SC, mod_id=sid)
    grads = torch.autograd.grad([x_out, y], dev, [dx_out.cuda(), dy.cuda()])
    pvl.device_error()

    ids = sid.cpu().long()
    ref = [t.double().requires_grad_() for t in (x, q, k, v, gate, shift, scale, wq, wk)]
    X, Q, K, V, GA, SH, SC, WQ, WK = ref
    ang = torch.from_numpy(oracle.rotary_angles(pos.cpu().numpy(), np.concatenate(
        [10000.0 ** (-np.arange(n) / n) for n in sections]), sections))[:, :, None]

    def rot(t, w):
        t = t / (t.pow(2).mean(2, keepdim=True) + 1e-6).sqrt() * w
        a, b = heads(t).chunk(2, dim=3)
        return torch.cat([a * ang.cos() - b * ang.sin(), a * ang.sin() + b * ang.cos()], dim=3)

    mask = (ids[:, :, None] == ids[:, None, :]) & (ids >= 0)[:, :, None]
    s = torch.einsum("blhd,bmhd->bhlm", rot(Q, WQ), rot(K, WK)) / D ** 0.5
    p = torch.softmax(s.masked_fill(~mask[:, None], -1e30), -1) * mask[:, None]
    o = torch.einsum("bhlm,bmhd->blhd", p, heads(V)).reshape(B, L, W)
    live, row = (ids >= 0)[..., None], ids.clamp(min=0)
    xo = torch.where(live, X + GA[row] * o, X)
    c = xo - xo.mean(2, keepdim=True)
    yo = torch.where(live, c / (c.pow(2).mean(2, keepdim=True) + 1e-6).sqrt() * (1 + SC[row]) + SH[row], 0.0)
    want = torch.autograd.grad([xo, yo], ref, [dx_out.double(), dy.double()])
    for name, u, w in zip("x_out y x q k v gate shift scale wq wk".split(), (x_out, y, *grads), (xo, yo, *want)):
        off = torch.linalg.norm(u.detach().cpu().double() - w) / torch.linalg.norm(w.detach())
        assert off <= 2.0 ** -5, f"{name}: relative error {off:.3e}"
