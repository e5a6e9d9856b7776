"""pack_preference_* and pack_policy_* against the fp64 oracle (GPU).

Tolerances, from the arithmetic.  A token's value is rounded once to 2^-40 and
then summed exactly; a token's terms are fp32: exp 2 ulp with its argument
rounded once (relative 2^-22 and 2^-24 |d|), products 2^-24 each: 2^-20 (1 + |d|)
of the term covers them.  exp f - f - 1 by the formula (|f| >= 0.5) carries 2^-22
of exp f + |f| + 1.  Losses of pairs: the argument x is rounded to fp32 (twice: D
to pairs, beta) and the losses are 1-Lipschitz: 2^-22 (1 + |x|).  Whether a ratio
is clipped is decided to 2^-48 on both sides."""

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


def pack(B, L, K, seed, prompt=True):
    """int32 [B, L] ids of K episodes a row, some of them empty, with prompts and tails of -1."""
    rng = np.random.default_rng(seed)
    ids = np.full((B, L), -1, dtype=np.int32)
    for b in range(B):
        cuts = np.sort(rng.integers(0, L + 1, size=K + 1))
        for k in range(K):
            start = cuts[k] + (int(rng.integers(0, (cuts[k + 1] - cuts[k]) // 3 + 1)) if prompt else 0)
            ids[b, start:cuts[k + 1]] = b * K + k
    return ids


def scattered(B, L, E, seed):
    """Ids in no order at all."""
    return np.random.default_rng(seed).integers(-1, E, size=(B, L)).astype(np.int32)


LAYOUTS = [("one token", lambda: np.zeros((1, 1), np.int32), 1), ("three tokens", lambda: np.array([[0, -1, 1]], np.int32), 2),
           ("odd", lambda: pack(3, 1001, 4, 1), 12), ("one episode", lambda: np.zeros((2, 5000), np.int32), 1),
           ("rows", lambda: np.repeat(np.arange(4, dtype=np.int32)[:, None], 2281, 1), 4),
           ("short episodes", lambda: pack(4, 4096, 300, 2), 1200), ("scattered", lambda: scattered(2, 3001, 50, 3), 50),
           ("64k", lambda: pack(1, 65536, 7, 4), 7), ("none", lambda: np.full((2, 70), -1, np.int32), 3)]


def floats(shape, seed, mul=1.0):
    return torch.from_numpy((np.random.default_rng(seed).normal(size=shape) * mul).astype(np.float32)).cuda()


def spoil(t, ids):
    """Infinities and NaN where no token takes part."""
    t = t.clone()
    off = torch.from_numpy(ids < 0).cuda()
    t[off] = float("nan")
    t.view(-1)[::2][off.view(-1)[::2]] = -math.inf
    return t


def check_preference(pvl, ids, E, pairs, seed=0, ref=True, mul=0.3, **how):
    lp, rf = floats(ids.shape, seed), floats(ids.shape, seed + 1, mul)
    rf = lp + rf if ref else None
    sid, pr = torch.from_numpy(ids).cuda(), torch.from_numpy(np.asarray(pairs, dtype=np.int32)).cuda()
    out = pvl.pack_preference_fwd(spoil(lp, ids), None if rf is None else spoil(rf, ids), sid, pr, E, **how)
    up = torch.tensor([1.7], device="cuda")
    d = pvl.pack_preference_bwd(up, out.coef, sid)
    pvl.device_error()
    loss, rewards, coef, grad = ob.preference(lp.cpu(), None if rf is None else rf.cpu(), ids, pairs, E, **how)
    beta, kind = how.get("beta", 0.1), how.get("kind", "sigmoid")
    live = np.asarray(pairs).min(1) >= 0
    x = (rewards[live][:, 0] - rewards[live][:, 1]) / beta - how.get("margin", 0.0)
    off = 2.0 ** -40 * ids.size                                      # of a sum
    if kind == "squared":
        miss = np.abs(x - 0.5 / beta)
        tol_loss, slope = 2.0 ** -22 * (miss ** 2) + 2 * miss * off, 2 * miss * 2.0 ** -22 + 2 * off
    else:
        tol_loss, slope = 2.0 ** -22 * (1 + np.abs(beta * x)) + beta * off, np.full(x.shape, beta * (2.0 ** -20 + off))
    assert abs(out.loss.item() - loss) <= (tol_loss.mean() if live.any() else 0.0) + 2.0 ** -23 * abs(loss)
    got = out.rewards.double().cpu().numpy()
    assert (np.abs(got - rewards) <= 2.0 ** -22 * np.abs(rewards) + beta * off).all() and not got[~live].any()
    tol = np.zeros(E)
    for (c, r), s in zip(np.asarray(pairs)[live], slope):
        tol[c] += s
        tol[r] += s
    tol = tol / max(1, live.sum()) + 2.0 ** -22 * np.abs(coef)
    if how.get("mean"):
        n = np.array([max(1, (ids == e).sum()) for e in range(E)])
        tol = tol / n + 2.0 ** -22 * np.abs(coef)
    assert (np.abs(out.coef.double().cpu().numpy() - coef) <= tol).all()
    gd = d.double().cpu().numpy()
    assert not gd[ids < 0].any()
    want = np.where(ids >= 0, 1.7 * out.coef.double().cpu().numpy()[np.maximum(ids, 0)], 0.0)
    assert (np.abs(gd - want) <= 2.0 ** -22 * np.abs(want)).all()
    return out, d


@pytest.mark.parametrize("name,make,E", LAYOUTS, ids=[v[0] for v in LAYOUTS])
@pytest.mark.parametrize("mean", [False, True])
def test_preference_layouts(pvl, name, make, E, mean):
    rng = np.random.default_rng(7)
    ids = make()
    pairs = rng.integers(0, E, size=(max(1, 2 * E), 2))
    check_preference(pvl, ids, E, pairs, mean=mean, beta=0.05, smoothing=0.1)


@pytest.mark.parametrize("kind", ["sigmoid", "squared", "hinge"])
@pytest.mark.parametrize("ref", [True, False])
def test_preference_kinds(pvl, kind, ref):
    ids = pack(2, 900, 10, 8)
    pairs = np.random.default_rng(9).integers(-1, 20, size=(33, 2))      # some left out, some against themselves
    for beta, margin in ((0.1, 0.0), (2.0, 0.3)):
        check_preference(pvl, ids, 20, pairs, ref=ref, kind=kind, beta=beta, margin=margin, mean=kind == "squared")


def test_preference_no_pair_and_the_same_pair_often(pvl):
    ids = pack(1, 300, 3, 10)
    out, d = check_preference(pvl, ids, 3, [[-1, 0], [1, -1], [-1, -1]])
    assert out.loss.item() == 0.0 and not d.any()
    check_preference(pvl, ids, 3, [[0, 1]] * 3000 + [[1, 0]] * 1000)
    out, d = check_preference(pvl, ids, 3, [[1, 1]] * 5)
    assert not d.any()


def test_preference_far_apart(pvl):
    """A pair whose margin is won by far: its factor is small and still right; the lost one saturates."""
    ids = torch.arange(2, dtype=torch.int32, device="cuda").repeat_interleave(10).view(1, -1)
    for gap in (5.0, 20.0, 35.0, 80.0):
        lp = torch.zeros(1, 20, device="cuda")
        lp[0, 0] = gap
        for beta in (1.0, 1e-3):
            out = pvl.pack_preference_fwd(lp / beta, None, ids, torch.tensor([[0, 1]], dtype=torch.int32, device="cuda"), 2, beta=beta)
            want = beta * math.exp(-gap) / (1 + math.exp(-gap))
            # relative to exp(-x), what x is off by: four roundings of it (h, beta, their product, a logit's own) of at
            # most 2^-24 |x| each, and 2^-19 for exp and the quotient; in units of 2^-80: exact to 2^-81 beta
            rel = 2.0 ** -22 * (8 + gap)
            tol = rel * want + beta * 2.0 ** -80
            assert abs(out.coef[0].item() + want) <= tol and abs(out.coef[1].item() - want) <= tol
            assert out.loss.item() == pytest.approx(math.log1p(math.exp(-gap)), rel=rel)
            lost = pvl.pack_preference_fwd(lp / beta, None, ids, torch.tensor([[1, 0]], dtype=torch.int32, device="cuda"), 2, beta=beta)
            assert lost.loss.item() == pytest.approx(gap + math.log1p(math.exp(-gap)), rel=2.0 ** -21)


def test_preference_values_that_are_not_finite_or_large(pvl):
    """A lowest-value log-probability saturates its pair, infinities of both sides give NaN, other pairs are untouched."""
    ids = torch.arange(4, dtype=torch.int32, device="cuda").repeat_interleave(10).view(1, -1)
    lp = torch.full((1, 40), -1.0, device="cuda")
    low = torch.finfo(torch.float32).min
    lp[0, 3] = low
    pairs = torch.tensor([[0, 1], [1, 0], [2, 3]], dtype=torch.int32, device="cuda")
    for kind in ("sigmoid", "hinge"):
        out = pvl.pack_preference_fwd(lp, None, ids, pairs, 4, kind=kind)
        want = torch.tensor([[0.1 * low, -1.0], [-1.0, 0.1 * low], [-1.0, -1.0]])
        assert torch.allclose(out.rewards.cpu(), want, rtol=1e-6)
        assert out.loss.item() == pytest.approx(-0.1 * low / 3, rel=1e-6)
        own = 0.05 if kind == "sigmoid" else 0.1
        assert torch.allclose(out.coef.cpu(), torch.tensor([-0.1 / 3, 0.1 / 3, -own / 3, own / 3]), rtol=1e-6)
    squared = pvl.pack_preference_fwd(lp, None, ids, pairs, 4, kind="squared")
    assert squared.loss.item() == math.inf
    both = -2.0 * abs(low) / 3 * 2      # the sum of the two lost pairs' derivatives passes the largest fp32
    assert squared.coef[0].item() in (both, -math.inf) and torch.isfinite(squared.coef[2:]).all()
    lp[0, 4] = -math.inf
    out = pvl.pack_preference_fwd(lp, None, ids, pairs, 4)
    assert out.rewards[0, 0] == -math.inf and torch.isfinite(out.coef).all() and out.loss.item() == math.inf
    lp[0, 5] = math.inf
    out = pvl.pack_preference_fwd(lp, None, ids, pairs, 4)
    assert torch.isnan(out.rewards[0, 0]) and torch.isnan(out.coef[:2]).all() and torch.isfinite(out.coef[2:]).all()


@pytest.mark.parametrize("gap", [1, 40, 5000])
def test_sums_do_not_cancel(pvl, gap):
    """1e30, 1, -1e30 in one episode, in one thread and in many: the 1 is left."""
    ids = torch.zeros(1, 2 * gap + 1, dtype=torch.int32, device="cuda")
    ids[0, 1::2] = 0 if gap == 1 else 1
    lp = torch.zeros(ids.shape, device="cuda")
    lp[0, 0], lp[0, 2 * gap] = 1e30, -1e30
    lp[0, 1 if gap == 1 else 2 * (gap // 2)] += 1.0
    out = pvl.pack_preference_fwd(lp, None, ids, torch.tensor([[0, 0]], dtype=torch.int32, device="cuda"), 2, beta=1.0)
    assert out.rewards[0, 0].item() == 1.0


def check_policy(pvl, ids, E, adv_tokens, seed=0, old=True, ref=True, spread=0.2, **how):
    lp = floats(ids.shape, seed)
    ol = lp + floats(ids.shape, seed + 1, spread) if old else None
    rf = lp + floats(ids.shape, seed + 2, 0.6) if ref else None
    adv = floats(ids.shape if adv_tokens else (E,), seed + 3)
    adv.view(-1)[::5] = 0.0
    sid = torch.from_numpy(ids).cuda()
    args = [spoil(lp, ids), None if ol is None else spoil(ol, ids), spoil(adv, ids) if adv_tokens else adv]
    rs = None if rf is None else spoil(rf, ids)
    out = pvl.pack_policy_fwd(*args, sid, E, ref_logp=rs, **how)
    up = torch.tensor([1.7], device="cuda")
    bw = {k: v for k, v in how.items() if k != "mean"}
    d = pvl.pack_policy_bwd(up, *args, sid, out.coef, ref_logp=rs, **bw)
    pvl.device_error()
    host = [None if t is None else t.cpu() for t in (lp, ol, adv)]
    loss, kl, share, grad = ob.policy(*host, ids, E, ref_logp=None if rf is None else rf.cpu(), **how)
    ok = ids >= 0
    n = np.array([(ids == e).sum() for e in range(E)], dtype=np.float64)
    weight = np.ones(E) / max(1, n.sum()) if how.get("mean", "token") == "token" else 1 / (np.maximum(n, 1) * max(1, (n > 0).sum()))
    w = np.where(ok, weight[np.maximum(ids, 0)], 0.0)
    a = adv.double().cpu().numpy()
    a = np.abs(np.where(ok, a if adv_tokens else a[np.maximum(ids, 0)], 0.0))
    r = 4.0 if old else 1.0                                         # exp(6 x 0.2) at most
    f = np.zeros(ids.shape) if rf is None else np.abs(rf.double().cpu().numpy() - lp.double().cpu().numpy())
    ef = np.exp(f) if rf is not None else np.zeros(ids.shape)
    klw = how.get("kl_weight", 0.0)
    tol_kl = 2.0 ** -21 * (w * np.where(f < 0.5, f * f, ef + f + 1)).sum() + 2.0 ** -40
    tol = 2.0 ** -19 * (w * r * a).sum() + klw * tol_kl + 2.0 ** -22 * abs(loss) + 2.0 ** -40
    assert abs(out.loss.item() - loss) <= tol, (out.loss.item(), loss, tol)
    assert abs(out.stats[0].item() - kl) <= tol_kl + 2.0 ** -22 * kl
    assert abs(out.stats[1].item() - share) <= 2.0 ** -23 * share
    gd = d.double().cpu().numpy()
    assert not gd[~ok].any()
    slack = 2.0 ** -19 * w * (r * a + klw * (1 + f) * np.maximum(ef - 1, 0)) * 1.7
    assert (np.abs(gd - 1.7 * grad) <= slack + 1e-38).all()
    return out, d


@pytest.mark.parametrize("name,make,E", LAYOUTS, ids=[v[0] for v in LAYOUTS])
@pytest.mark.parametrize("mean", ["token", "episode"])
@pytest.mark.parametrize("ratio", ["token", "episode"])
def test_policy_layouts(pvl, name, make, E, mean, ratio):
    wide = 0.1 if ratio == "token" else 0.005
    for adv_tokens in ((True, False) if ratio == "token" else (False,)):
        check_policy(pvl, make(), E, adv_tokens, mean=mean, ratio=ratio, clip_low=wide, clip_high=1.5 * wide, kl_weight=0.1)


@pytest.mark.parametrize("old", [True, False])
@pytest.mark.parametrize("ref", [True, False])
def test_policy_optional_inputs(pvl, old, ref):
    ids = pack(2, 777, 5, 11)
    for ratio in ("token", "episode"):
        for klw in ((0.0, 0.3) if ref else (0.0,)):
            out, d = check_policy(pvl, ids, 10, False, old=old, ref=ref, ratio=ratio, kl_weight=klw)
            if not old:
                assert out.stats[1].item() == 0.0


def test_policy_values_that_are_not_finite(pvl):
    """A ratio past fp32 counts as clipped with A > 0, is infinite with A < 0 and gives 0 with A = 0."""
    ids = torch.zeros(1, 3, dtype=torch.int32, device="cuda")
    lp, old = torch.zeros(1, 3, device="cuda"), torch.tensor([[-200.0, 0.0, 0.0]], device="cuda")
    for a, loss, grad in ((1.0, -1.2, 0.0), (0.0, 0.0, 0.0), (-1.0, math.inf, math.inf)):
        adv = torch.tensor([[a, 0.0, 0.0]], device="cuda")
        out = pvl.pack_policy_fwd(lp, old, adv, ids, 1)
        d = pvl.pack_policy_bwd(None, lp, old, adv, ids, out.coef)
        assert out.loss.item() == pytest.approx(loss / 3, rel=1e-6) and d[0].tolist() == [grad, 0.0, 0.0]
    # a divergence that is infinite is no part of a loss that does not weigh it
    ref = torch.tensor([[200.0, 0.0, 0.0]], device="cuda")
    out = pvl.pack_policy_fwd(lp, lp, torch.ones(1, 3, device="cuda"), ids, 1, ref_logp=ref)
    assert out.loss.item() == -1.0 and out.stats[0].item() == math.inf
    assert torch.isfinite(pvl.pack_policy_bwd(None, lp, lp, torch.ones(1, 3, device="cuda"), ids, out.coef, ref_logp=ref)).all()
    # a log-probability of -inf: an infinite divergence, no NaN; one of the reference's too
    gone = torch.tensor([[-math.inf, 0.0, 0.0]], device="cuda")
    for a, b in ((gone, lp), (lp, gone)):
        out = pvl.pack_policy_fwd(a, torch.zeros_like(lp), torch.ones(1, 3, device="cuda"), ids, 1, ref_logp=b, kl_weight=0.1)
        assert out.loss.item() == math.inf and out.stats[0].item() == math.inf
    # a NaN stays in its token's gradient and reaches the loss
    lp[0, 1] = math.nan
    out = pvl.pack_policy_fwd(lp, torch.zeros_like(lp), torch.ones(1, 3, device="cuda"), ids, 1)
    d = pvl.pack_policy_bwd(None, lp, torch.zeros_like(lp), torch.ones(1, 3, device="cuda"), ids, out.coef)
    assert math.isnan(out.loss.item()) and torch.isnan(d[0]).tolist() == [False, True, False]


def test_large_terms(pvl):
    """Terms of 2^11 and more, next to small ones."""
    ids = pack(1, 3000, 2, 21, prompt=False)
    lp = floats(ids.shape, 22)
    old = lp.clone()
    old[0, ::50] -= 10.0                                            # ratios of 22026
    adv = -floats(ids.shape, 23).abs() - 0.1
    out = pvl.pack_policy_fwd(lp, old, adv, torch.from_numpy(ids).cuda(), 2)
    loss = ob.policy(lp.cpu(), old.cpu(), adv.cpu(), ids, 2)[0]
    assert out.loss.item() == pytest.approx(loss, rel=2.0 ** -18)


def test_divergence_of_near_policies(pvl):
    """exp f - f - 1 of small f, where the formula would leave nothing."""
    f = torch.tensor([[1e-4, 1e-3, 1e-2, 0.1, 0.49, 0.51, -0.49, -1e-3, 40.0]], device="cuda")
    ids = torch.zeros(f.shape, dtype=torch.int32, device="cuda")
    for i in range(f.shape[1]):
        one = torch.full_like(ids, -1)
        one[0, i] = 0
        out = pvl.pack_policy_fwd(torch.zeros_like(f), None, torch.zeros_like(f), one, 1, ref_logp=f, kl_weight=1.0)
        x = float(f[0, i])
        want = x * x / 2 + x ** 3 / 6 + x ** 4 / 24 if abs(x) <= 1e-3 else math.expm1(x) - x
        assert abs(out.stats[0].item() - want) <= want * (2.0 ** -20 if abs(x) < 0.5 else 2.0 ** -19) + 2.0 ** -47     # summed in units of 2^-46


def test_unaligned_tokens_and_outputs(pvl):
    """Tokens that start off a 16-byte boundary, as parts of longer buffers."""
    ids = pack(1, 1500, 6, 12)
    sid = torch.from_numpy(ids).cuda().view(-1)
    lp, old, adv = (floats((1500,), 20 + i) for i in range(3))
    a = pvl.pack_policy_fwd(lp, old, adv, sid, 6)
    ga = pvl.pack_policy_bwd(None, lp, old, adv, sid, a.coef)

    def shift(t):
        out = torch.empty(1503, dtype=t.dtype, device="cuda")
        out[3:] = t
        return out[3:]

    s = [shift(t) for t in (lp, old, adv, sid)]
    b = pvl.pack_policy_fwd(*s, 6)
    buf = torch.full((1505,), 7.0, device="cuda")
    gb = pvl.pack_policy_bwd(None, *s, b.coef, dlogp=buf[3:1503])
    assert torch.equal(a.loss, b.loss) and torch.equal(ga, gb)
    assert (buf[:3] == 7).all() and (buf[1503:] == 7).all()


def test_ids_past_the_episodes(pvl):
    """Left out and reported; the pairs too."""
    from packed_variable_length_gb300.api import PVL_ERR_INVALID_ARG
    ids = torch.tensor([[0, 0, 1, 1, 2, 9]], dtype=torch.int32, device="cuda")
    lp = torch.randn(1, 6, device="cuda")
    pairs = torch.tensor([[0, 1], [0, 5]], dtype=torch.int32, device="cuda")
    out = pvl.pack_preference_fwd(lp, None, ids, pairs[:1], 2)
    assert pvl.device_error(raise_on_error=False)[0] == PVL_ERR_INVALID_ARG
    want = pvl.pack_preference_fwd(lp[:, :4].contiguous(), None, ids[:, :4].contiguous(), pairs[:1], 2)
    assert pvl.device_error(raise_on_error=False)[0] == 0
    assert torch.equal(out.loss, want.loss)
    both = pvl.pack_preference_fwd(lp[:, :4].contiguous(), None, ids[:, :4].contiguous(), pairs, 2)
    with pytest.raises(pvl.PvlError):
        pvl.device_error()
    assert torch.equal(both.loss, want.loss) and not both.rewards[1].any()
    d = pvl.pack_preference_bwd(None, out.coef, ids)
    assert not d[0, 4:].any()
    adv = torch.randn(2, device="cuda")
    p = pvl.pack_policy_fwd(lp, lp - 0.1, adv, ids, 2)
    with pytest.raises(pvl.PvlError):
        pvl.device_error()
    q = pvl.pack_policy_fwd(lp[:, :4].contiguous(), lp[:, :4] - 0.1, adv, ids[:, :4].contiguous(), 2)
    assert torch.equal(p.loss, q.loss)
    assert not pvl.pack_policy_bwd(None, lp, lp - 0.1, adv, ids, p.coef)[0, 4:].any()


def test_same_bits_twice(pvl):
    """Whatever order the blocks finish in, also where an episode is spread over all of them."""
    for ids, E in ((scattered(8, 20001, 5, 13), 5), (pack(8, 32768, 64, 14), 512)):
        lp, rf = floats(ids.shape, 15), floats(ids.shape, 16)
        sid = torch.from_numpy(ids).cuda()
        pairs = torch.from_numpy(np.random.default_rng(17).integers(0, E, size=(500, 2)).astype(np.int32)).cuda()
        adv = floats((E,), 18)
        a = pvl.pack_preference_fwd(lp, rf, sid, pairs, E)
        p = pvl.pack_policy_fwd(lp, rf, adv, sid, E, ref_logp=rf, kl_weight=0.1, mean="episode")
        for _ in range(20):
            assert all(torch.equal(u, v) for u, v in zip(a, pvl.pack_preference_fwd(lp, rf, sid, pairs, E)))
            again = pvl.pack_policy_fwd(lp, rf, adv, sid, E, ref_logp=rf, kl_weight=0.1, mean="episode")
            assert all(torch.equal(u, v) for u, v in zip(p, again))


def test_most_tokens_and_many_episodes(pvl):
    """2^23 tokens of 65,536 episodes, id by id in turn: every token is a run of its own."""
    N, E = 1 << 23, 1 << 16
    sid = (torch.arange(N, device="cuda", dtype=torch.int32) % E)
    lp = (torch.arange(N, device="cuda") // E).float()              # 0 .. 127 in each episode
    pairs = torch.stack([torch.arange(E - 1), torch.arange(1, E)], 1).int().cuda()
    out = pvl.pack_preference_fwd(lp, None, sid, pairs, E, beta=1.0)
    pvl.device_error()
    assert (out.rewards == 127 * 64).all() and out.loss.item() == pytest.approx(math.log(2), rel=1e-6)
    ends = out.coef[[0, -1]].cpu() * (E - 1)
    assert torch.allclose(ends, torch.tensor([-0.5, 0.5]), rtol=1e-5) and out.coef[1:-1].abs().max() < 1e-10
    p = pvl.pack_policy_fwd(lp, lp, torch.ones(E, device="cuda"), sid, E, mean="episode", ratio="episode")
    assert p.loss.item() == -1.0


@pytest.mark.parametrize("N", [127, 128, 129, 2047, 2048, 2049, 140000])
def test_both_sides_of_a_warp_and_of_a_block(pvl, N):
    """A warp takes 128 tokens, a block 2048."""
    ids = pack(1, N, 9, N)
    pairs = np.random.default_rng(N).integers(0, 9, size=(20, 2))
    check_preference(pvl, ids, 9, pairs, mean=True)
    check_policy(pvl, ids, 9, True, kl_weight=0.1)
    check_policy(pvl, ids, 9, False, ratio="episode", mean="episode", clip_low=0.01, clip_high=0.01)
