"""Rotary positions where a block holds several teams and a team takes many tokens, against the formulas in fp64 (GPU).

Tolerances are those of test_gpu_rotary: 2^-15 of a pair's magnitude forward, 2^-14 of the gradient's two terms, and
2^-13 of the sum of magnitudes for a weight's gradient, whose chains stay below 2^8 here too (a team's tokens, at most
220, then 32 rows of partial sums at a time)."""

import pytest
import torch

pytestmark = pytest.mark.gpu
STEP = torch.finfo(torch.bfloat16).eps / 2
EPS = 1e-5


@pytest.fixture(scope="module")
def pvl(cuda_ok):
    import packed_variable_length_gb300 as p
    return p


def sides(v, layout):
    """First and second features of the pairs of v's last dimension."""
    n = v.shape[-1] // 2
    return (v[..., :n], v[..., n:]) if layout == "half" else (v[..., 0::2], v[..., 1::2])


def joined(a, b, layout):
    return torch.cat([a, b], -1) if layout == "half" else torch.stack([a, b], -1).flatten(-2)


def turned(v, angle, R, layout):
    a, b = sides(v[..., :R], layout)
    c, s = angle.cos(), angle.sin()
    return torch.cat([joined(a * c - b * s, a * s + b * c, layout), v[..., R:]], -1)


def pair_magnitude(v, R, layout):
    a, b = sides(v[..., :R], layout)
    m = torch.hypot(a, b)
    return torch.cat([joined(m, m, layout), v[..., R:].abs()], -1)


def near(name, got, ref, mag, step=STEP):
    got = got.double()
    assert bool(got.isfinite().all()), name
    err = (got - ref).abs() - step * ref.abs() - mag
    worst = float(err.max())
    assert worst <= 0, f"{name}: {int((err > 0).sum())} values out of tolerance, worst by {worst:.3e}"


def check(pvl, L, H, Hk, D, R, layout, norm, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def heads(n):
        return torch.randn(1, L, n, D, generator=g, device="cuda").to(torch.bfloat16)

    wide = norm == "token"
    q, k, dq, dk = heads(H), heads(Hk), heads(H), heads(Hk)
    wq, wk = (1 + 0.2 * torch.randn(n * D if wide else D, generator=g, device="cuda") for n in (H, Hk))
    pos = torch.randint(-100, 400, (1, L), generator=g, device="cuda", dtype=torch.int32)
    plan = pvl.rotary_plan(R, layout=layout)
    out = pvl.pack_rotary_fwd(q, k, pos, plan, norm, wq, wk, eps=EPS)
    grads = pvl.pack_rotary_bwd(dq, dk, pos, plan, norm, q, k, wq, wk, eps=EPS)
    pvl.device_error()
    freqs = 10000.0 ** (-torch.arange(R // 2, device="cuda", dtype=torch.float64) / (R // 2))
    angle = (pos.double()[..., None] * freqs)[:, :, None]
    over = (2, 3) if wide else (3,)
    for name, x, o, dout, w, dx, dw in (("q", q, out[0], dq, wq, grads[0], grads[2]),
                                        ("k", k, out[1], dk, wk, grads[1], grads[3])):
        x, w = x.double(), w.double().view(-1, D)
        r = 1.0 / (x.square().mean(over, keepdim=True) + EPS).sqrt()
        xh = x * r
        ref = turned(xh * w, angle, R, layout)
        near(name, o, ref, 2.0 ** -15 * pair_magnitude(ref, R, layout))
        up = turned(dout.double(), -angle, R, layout)
        g0 = pair_magnitude(up, R, layout)
        sums = (0, 1) if wide else (0, 1, 2)
        near("dw" + name, dw, (up * xh).sum(sums).flatten(), 2.0 ** -13 * (g0 * xh.abs()).sum(sums).flatten(),
             step=2.0 ** -24)
        ref = r * (up * w - xh * (up * w * xh).mean(over, keepdim=True))
        g0 = g0 * w.abs()
        near("d" + name, dx, ref, 2.0 ** -14 * r * (g0 + xh.abs() * (g0 * xh.abs()).mean(over, keepdim=True)))
    for _ in range(10):
        for u, v in zip(grads, pvl.pack_rotary_bwd(dq, dk, pos, plan, norm, q, k, wq, wk, eps=EPS)):
            assert torch.equal(u, v)


@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("L", [20001, 65535])
@pytest.mark.parametrize("dims", [(8, 4, 128, 128), (2, 2, 128, 128), (4, 4, 128, 96), (16, 8, 64, 64), (1, 1, 64, 64),
                                  (12, 12, 128, 128), (6, 2, 72, 72)])
def test_norm_over_the_token(pvl, dims, L, layout):
    """Teams of part of a warp, of one and of two, none of which divides the tokens."""
    check(pvl, L, *dims, layout, "token", seed=L)


@pytest.mark.parametrize("dims", [(8, 4, 128, 128), (1, 1, 64, 64), (12, 12, 128, 128), (6, 2, 72, 72)])
def test_norm_per_head(pvl, dims):
    check(pvl, 20001, *dims, "half", "head", seed=1)


@pytest.mark.parametrize("norm", ["head", "token"])
def test_one_head_a_thread_and_several(pvl, norm):
    """The same heads on both sides of the token count from which a thread takes several of them."""
    for L in (303, 304, 305, 309, 5001):
        check(pvl, L, 5, 3, 128, 128, "half", norm, seed=L)


def test_a_refused_call_leaves_no_error_behind(pvl):
    """A backward whose token does not fit a block is refused, and the calls after it succeed."""
    L, H, Hk, D = 9, 128, 8, 128
    q, k = (torch.randn(1, L, n, D, device="cuda").to(torch.bfloat16) for n in (H, Hk))
    pos = torch.arange(L, dtype=torch.int32, device="cuda")[None]
    plan = pvl.rotary_plan(D)
    with pytest.raises(pvl.PvlError):
        pvl.pack_rotary_bwd(q, k, pos, plan, "token", q, k)
    got = pvl.pack_build_positions([[3]], 3, L)
    assert got.flatten().tolist() == list(range(L))
    pvl.pack_rotary_fwd(q, k, pos, plan, "token")       # the forward does fit
    x = torch.randn(1, 4, 64, device="cuda").to(torch.bfloat16)
    pvl.adaln_fwd(x, torch.zeros(1, 64, device="cuda"), torch.zeros(1, 64, device="cuda"))
    pvl.adaln_residual_fwd(x)
    pvl.device_error()


@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("H,Hk,D", [(100, 32, 128), (44, 8, 232), (40, 8, 220), (40, 8, 194), (44, 4, 254)])
def test_the_widest_tokens(pvl, H, Hk, D, layout):
    """As many heads as the norm over the token holds, backward too, at every width of vectors."""
    for L in (7, 700):
        check(pvl, L, H, Hk, D, D, layout, "token", seed=D)
