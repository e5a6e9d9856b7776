"""pack_logprob_fwd / pack_logprob_bwd against the fp64 oracle (GPU).

Tolerances, from the arithmetic.  exp2 of a difference: its argument carries
three fp32 roundings relative to |t|, ex2 2^-22; weighted by exp(-|t|) these
are at most 2^-21.5 of the largest term.  A thread adds up to V / 8 terms
(2^-24 each).  So the sum's relative error is at most rel = 2^-20 + V 2^-27 (eight
threads a row, up to 512 logits), 2^-20 + V 2^-29 (a warp) and 2^-20 + V 2^-32
(a block); rel_of takes the number of threads.  logp and lse add roundings
relative to themselves and to the maximum; the entropy weights the errors by up
to log V; the gradient's probability carries rel and the roundings of z and lse,
and is rounded once to the logits' type.  ex2 gives 0 for probabilities below the
smallest normal fp32 number, 2^-126, so the gradient is off by up to that times what
multiplies the probability, and by it where the product is below it."""

import math

import numpy as np
import pytest
import torch

from oracle import objectives as ob

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def pvl(cuda_ok):
    import packed_variable_length_gb300 as p
    return p


def rel_of(V):
    return 2.0 ** -20 + V / (8 if V <= 520 else 32 if V <= 2056 else 256) * 2.0 ** -24


def check(pvl, x, t, ids=None, T=1.0, ent=True, seed=0, at=None):
    """Forward and backward of logits x (a CUDA view), rows `at` (b, l) compared; the others for being finite."""
    B, L, V = x.shape
    g = torch.Generator().manual_seed(seed)
    up, ue = torch.randn(B, L, generator=g).cuda(), torch.randn(B, L, generator=g).cuda()
    logp, lse, h = pvl.pack_logprob_fwd(x, t, ids, temperature=T, entropy=ent)
    assert (h is None) == (not ent)
    d = pvl.pack_logprob_bwd(up, x, t, lse, ids, temperature=T, ent=h, dent=ue if ent else None)
    torch.cuda.synchronize()
    assert d.shape == x.shape and d.dtype == x.dtype
    hx, ht = x.cpu(), t.cpu().numpy()
    valid = ob.valid_targets(ht, V, None if ids is None else ids.cpu().numpy())
    if at is not None:
        keep = np.zeros_like(valid)
        for b, l in at:
            keep[b, l] = True
        valid = valid & keep
    rl, rs, rh = ob.logprob(hx, ht, valid, T)
    rel = rel_of(V)
    got = [v.double().cpu().numpy() for v in (logp, lse)]
    top = np.where(valid, np.nan_to_num(hx.double().numpy(), neginf=0.0).max(2) / T, 0.0)
    tol = rel + 2.0 ** -22 * (np.abs(top) + np.abs(rs))
    assert (np.abs(got[0] - rl)[valid] <= (tol + 2.0 ** -22 * np.abs(rl))[valid]).all()
    assert (np.abs(got[1] - rs)[valid] <= tol[valid]).all()
    if ent:
        assert (np.abs(h.double().cpu().numpy() - rh)[valid] <= (rel * (4 + 2 * math.log(max(V, 2))) + 2.0 ** -22 * rh)[valid]).all()
    if at is None:
        for v in (logp, lse) + ((h,) if ent else ()):
            assert not v.cpu().numpy()[~valid].any()
        assert not d.cpu().float().numpy()[~valid].any()
    ref = ob.logprob_grad(hx, ht, valid, up.cpu(), ue.cpu() if ent else None, T)
    z = np.where(valid[..., None], hx.double().numpy() / T - rs[..., None], -np.inf)
    p = np.exp(z)
    unit = 2.0 ** -8 if x.dtype == torch.bfloat16 else 2.0 ** -23
    off = rel + 2.0 ** -22 * (np.abs(top) + np.abs(rs) + 2)
    zs = np.where(p > 0, np.abs(z), 0.0)
    slack = (p * (off[..., None] + 2.0 ** -22 * zs) + 2.0 ** -126) * (np.abs(up.double().cpu().numpy())[..., None] + (np.abs(
        ue.double().cpu().numpy())[..., None] * (zs + rh[..., None] + 2) if ent else 0.0)) / T
    err = np.abs(d.double().cpu().numpy() - ref)[valid]
    assert (err <= (unit * np.abs(ref) + slack)[valid] + 2.0 ** -126).all(), err.max()
    return logp, lse, h, d


def make(B, L, V, dtype, seed, mul=3.0, add=0.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = (torch.randn(B, L, V, generator=g, device="cuda") * mul + add).to(dtype)
    t = torch.randint(0, V, (B, L), generator=g, device="cuda", dtype=torch.int32)
    return x, t


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("V", [1, 2, 7, 8, 9, 63, 256, 257, 511, 519, 520, 521, 1000, 2047, 2048, 2056, 2057, 4099, 16383, 16384])
def test_sizes(pvl, V, dtype):
    """Both sides of every rule on V, in both types, odd rows at every alignment."""
    x, t = make(2, 9, V, dtype, V)
    check(pvl, x, t, seed=V, ent=V % 2 == 0)


@pytest.mark.parametrize("rows", [(1, 1), (4, 38), (153, 1)])
@pytest.mark.parametrize("dtype,V", [(torch.bfloat16, 16391), (torch.bfloat16, 32768), (torch.float32, 8193)])
def test_few_rows_of_many_logits(pvl, rows, dtype, V):
    """A cluster a row up to as many rows as SMs (152), and the block a row past it."""
    x, t = make(*rows, V, dtype, 3)
    check(pvl, x, t, at=[(0, 0), (rows[0] - 1, rows[1] - 1)])


@pytest.mark.parametrize("N,V,dtype", [(20000, 2, torch.bfloat16), (20000, 23, torch.bfloat16), (20000, 509, torch.bfloat16),
                                       (20000, 253, torch.float32), (1215, 256, torch.bfloat16), (1216, 256, torch.bfloat16), (5000, 1009, torch.bfloat16),
                                       (9727, 2048, torch.bfloat16), (9729, 2055, torch.bfloat16), (9729, 1027, torch.float32),
                                       (1215, 8191, torch.bfloat16), (1217, 8197, torch.bfloat16), (1217, 16391, torch.bfloat16),
                                       (1300, 8193, torch.float32), (50, 32768, torch.bfloat16), (52, 32768, torch.bfloat16),
                                       (200, 128001, torch.bfloat16), (3000, 33000, torch.bfloat16)])
def test_both_sides_of_the_rules_on_rows(pvl, N, V, dtype):
    """Many rows, against torch in 64 bits on the device; every thread of a row may add V / 8 terms."""
    x, t = make(1, N, V, dtype, N)
    up, ue = randn(1, N, seed=1), randn(1, N, seed=2)
    logp, lse, h = pvl.pack_logprob_fwd(x, t, entropy=True)
    d = pvl.pack_logprob_bwd(up, x, t, lse, ent=h, dent=ue)
    rel = 2.0 ** -20 + V / 8 * 2.0 ** -24
    unit = 2.0 ** -8 if dtype == torch.bfloat16 else 2.0 ** -23
    for i in range(0, N, 500):
        at = slice(i, i + 500)
        logs = torch.log_softmax(x[0, at].double(), 1)
        p = logs.exp()
        pick = t[0, at, None].long()
        top = x[0, at].double().abs().amax(1)
        s = torch.logsumexp(x[0, at].double(), 1)
        ent = -(p * logs).sum(1)
        tol = rel + 2.0 ** -22 * (top + s.abs())
        assert ((logp[0, at] - logs.gather(1, pick)[:, 0]).abs() <= tol + 2.0 ** -22 * logs.gather(1, pick)[:, 0].abs()).all()
        assert ((lse[0, at] - s).abs() <= tol).all()
        assert ((h[0, at] - ent).abs() <= rel * (4 + 2 * math.log(V)) + 2.0 ** -22 * ent).all()
        g, ge = up[0, at, None].double(), ue[0, at, None].double()
        want = -p * (g + ge * (logs + ent[:, None]))
        want.scatter_add_(1, pick, g)
        slack = p * (tol[:, None] + 2.0 ** -22 * (2 + logs.abs())) * (g.abs() + ge.abs() * (logs.abs() + ent[:, None] + 2))
        assert ((d[0, at].double() - want).abs() <= unit * want.abs() + slack + 2.0 ** -120).all()


def randn(*shape, seed):
    return torch.randn(*shape, generator=torch.Generator(device="cuda").manual_seed(seed), device="cuda")


def test_padding_targets_and_temperature(pvl):
    """Invalid tokens, by id and by target, hold NaN and infinities; int64 targets; temperatures."""
    for T in (0.25, 1.0, 3.0):
        for dtype in (torch.bfloat16, torch.float32):
            x, t = make(3, 17, 777, dtype, 5)
            ids = torch.zeros(3, 17, dtype=torch.int32, device="cuda")
            ids[0, 5:9] = -1
            ids[2] = -1
            t[1, 0], t[1, 1], t[1, 2] = -100, 777, 2 ** 31 - 1
            bad = (ids < 0) | (t < 0) | (t >= 777)
            x[bad] = float("nan")
            x[0, 5] = float("inf")
            check(pvl, x, t, ids, T)
            wide = t.long()
            wide[1, 2] = 2 ** 40
            wide[1, 0] = -2 ** 40
            a, b = pvl.pack_logprob_fwd(x, t, ids, temperature=T)[0], pvl.pack_logprob_fwd(x, wide, ids, temperature=T)[0]
            assert torch.equal(a, b)


def test_nothing_valid(pvl):
    x, t = make(2, 3, 300, torch.bfloat16, 6)
    ids = torch.full((2, 3), -1, dtype=torch.int32, device="cuda")
    logp, lse, h, d = check(pvl, x * float("nan"), t, ids)
    assert not logp.any() and not lse.any() and not h.any() and not d.any()


@pytest.mark.parametrize("V", [40, 600, 5000, 20000])
def test_banned_and_lowest_logits(pvl, V):
    """-inf and the type's lowest value in part of a row, a chosen banned token, one logit left, a common offset."""
    for dtype in (torch.bfloat16, torch.float32):
        x, t = make(1, 6, V, dtype, 7)
        low = torch.finfo(dtype).min
        x[0, 0, ::3] = -math.inf
        x[0, 1, 1:] = -math.inf
        x[0, 2] = low
        x[0, 3, 1::2] = low
        x[0, 4] += 300.0
        x[0, 5] -= 30000.0
        t[0] = torch.tensor([1, 0, 3, 0, 1, 2])
        check(pvl, x, t)
        t[0, 0] = 3                      # banned: probability 0
        logp, lse, h = pvl.pack_logprob_fwd(x, t, entropy=True)
        assert logp[0, 0] == -math.inf and torch.isfinite(h).all()
        d = pvl.pack_logprob_bwd(torch.ones_like(logp), x, t, lse, ent=h, dent=torch.ones_like(h))
        assert torch.isfinite(d).all() and d[0, 0, 3] == 1.0 and d[0, 0, 0] == 0.0


def test_rows_without_a_distribution(pvl):
    """As a log-softmax has it: only -inf, NaN, +inf."""
    for V in (40, 600, 20000):
        x, t = make(1, 3, V, torch.float32, 8)
        x[0, 0] = -math.inf
        x[0, 1, V // 2] = math.nan
        x[0, 2, V - 1] = math.inf
        logp, lse, h = pvl.pack_logprob_fwd(x, t, entropy=True)
        assert torch.isnan(logp).all() and torch.isnan(h).all() and lse[0, 0] == -math.inf


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("V", [37, 1001, 9000])
def test_strides(pvl, V, dtype):
    """A padded vocabulary, shifted tokens, a transposed batch, an odd start; gradients into views."""
    big, t = make(3, 8, V + 5, dtype, 9)
    for x in (big[..., :V], big[:, :-1, 3:3 + V], big.transpose(0, 1)[..., 1:1 + V], big[1:2, :, :V], big[:, 2:3, :V]):
        B, L = x.shape[:2]
        tt = t[:1, :1].expand(B, L).contiguous() % V
        want = check(pvl, x, tt)
        up = torch.Generator().manual_seed(0)
        up, ue = torch.randn(B, L, generator=up).cuda(), torch.randn(B, L, generator=up).cuda()
        out = torch.full((B, L + 1, V + 3), 7.0, dtype=dtype, device="cuda")
        turned = torch.full((L, B + 1, V + 3), 7.0, dtype=dtype, device="cuda")
        for buf, view in ((out, out[:, 1:, 2:2 + V]), (turned, turned[:, 1:, 2:2 + V].transpose(0, 1))):
            pvl.pack_logprob_bwd(up, x, tt, want[1], ent=want[2], dent=ue, dlogits=view)
            assert torch.equal(view, want[3])
            assert (buf[:, 0] == 7).all() and (buf[..., :2] == 7).all() and (buf[..., 2 + V:] == 7).all()


@pytest.mark.parametrize("V", [5, 300, 1111, 20001])
def test_gradient_over_the_logits(pvl, V):
    for dtype in (torch.bfloat16, torch.float32):
        x, t = make(2, 5, V, dtype, 10)
        t[0, 2] = -1
        logp, lse, _ = pvl.pack_logprob_fwd(x, t)
        up = torch.randn(2, 5, device="cuda")
        want = pvl.pack_logprob_bwd(up, x, t, lse)
        got = pvl.pack_logprob_bwd(up, x, t, lse, dlogits=x)
        assert got is x and torch.equal(x, want)


def test_upstream_gradients_of_padding_are_not_used(pvl):
    x, t = make(2, 5, 333, torch.float32, 14)
    ids = torch.tensor([[0, 0, -1, 0, -1], [1, 1, 1, 1, -1]], dtype=torch.int32, device="cuda")
    logp, lse, h = pvl.pack_logprob_fwd(x, t, ids, entropy=True)
    up, ue = torch.randn(2, 2, 5, device="cuda").unbind(0)
    want = pvl.pack_logprob_bwd(up, x, t, lse, ids, ent=h, dent=ue)
    for v in (up, ue, lse, h):
        v[ids < 0] = math.nan
    got = pvl.pack_logprob_bwd(up, x, t, lse, ids, ent=h, dent=ue)
    assert torch.equal(got, want) and not got[ids < 0].any()


def test_only_the_entropys_gradient(pvl):
    x, t = make(2, 5, 333, torch.float32, 11)
    logp, lse, h = pvl.pack_logprob_fwd(x, t, entropy=True)
    ue = torch.randn(2, 5, device="cuda")
    a = pvl.pack_logprob_bwd(None, x, t, lse, ent=h, dent=ue)
    b = pvl.pack_logprob_bwd(torch.zeros_like(ue), x, t, lse, ent=h, dent=ue)
    assert torch.equal(a, b)


def test_offsets_past_32_bits(pvl):
    """70,000 rows of 32,768 logits: 2.3 G elements; the last rows against the oracle, and against a copy of them."""
    N, V = 70000, 32768
    x = torch.zeros(1, N, V, dtype=torch.bfloat16, device="cuda")
    t = torch.zeros(1, N, dtype=torch.int32, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(12)
    x[0, -3:] = torch.randn(3, V, generator=g, device="cuda").bfloat16() * 4
    t[0, -3:] = torch.tensor([5, 100, V - 1], dtype=torch.int32)
    tail_x, tail_t = x[:, -3:].clone(), t[:, -3:].clone()     # x is overwritten below
    logp, lse, h, d = check(pvl, tail_x, tail_t)
    a, b, c = pvl.pack_logprob_fwd(x, t, entropy=True)
    # three rows go to a cluster each, many to a block each: other orders of the same sums
    for u, v in ((a, logp), (b, lse), (c, h)):
        assert torch.allclose(u[0, -3:], v[0], rtol=0, atol=4e-5)
    assert torch.allclose(a[0, :-3], torch.tensor(-math.log(V), device="cuda"), rtol=0, atol=4e-5)
    up, ue = torch.randn(2, 1, N, generator=g, device="cuda").unbind(0)
    got = pvl.pack_logprob_bwd(up, x, t, b, ent=c, dent=ue, dlogits=x)
    part = pvl.pack_logprob_bwd(up[:, -3:].contiguous(), tail_x, tail_t, b[:, -3:].contiguous(),
                                ent=c[:, -3:].contiguous(), dent=ue[:, -3:].contiguous())
    assert torch.equal(got[:, -3:], part)


def test_same_bits_twice(pvl):
    for V in (100, 1000, 30000):
        x, t = make(2, 50, V, torch.bfloat16, 13)
        first = pvl.pack_logprob_fwd(x, t, entropy=True)
        for _ in range(3):
            assert all(torch.equal(a, b) for a, b in zip(first, pvl.pack_logprob_fwd(x, t, entropy=True)))
