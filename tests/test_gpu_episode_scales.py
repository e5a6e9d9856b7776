"""Losses over episodes of small and large terms: sums keep what is small, and means of what is large are finite (GPU).

Tolerances: a token's value is rounded to 2^-80 (off by 2^-81) and then summed exactly; terms of the policy loss carry
2^-20 (1 + |d|) of themselves, the divergence's series 2^-20, both as derived beside the tests of ordinary values."""

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


def layout(kind, N=5000, E=6):
    """One episode a block, one a warp, one a lane, one a token; some tokens of none."""
    at = np.arange(N)
    ids = {"block": at // 2500, "warp": at // 128 % E, "lane": at // 4 % E, "token": at % E}[kind].astype(np.int32)
    ids[1000:1100] = -1
    return ids, E


@pytest.mark.parametrize("kind", ["block", "warp", "lane", "token"])
@pytest.mark.parametrize("mean", ["token", "episode"])
@pytest.mark.parametrize("size", [1e-3, 1e-6, 1e-9, 1e-14])
def test_small_advantages(pvl, kind, mean, size):
    """The loss of advantages 10^9 times smaller is 10^9 times smaller, as its gradient is."""
    ids, E = layout(kind)
    rng = np.random.default_rng(1)
    lp = torch.from_numpy(-rng.exponential(size=ids.shape).astype(np.float32)).cuda()
    old = lp + torch.from_numpy(rng.normal(size=ids.shape).astype(np.float32) * 0.1).cuda()
    adv = torch.from_numpy((rng.normal(size=ids.shape) * size).astype(np.float32)).cuda()
    sid = torch.from_numpy(ids).cuda()
    out = pvl.pack_policy_fwd(lp, old, adv, sid, E, mean=mean)
    pvl.device_error()
    want, _, share, _ = ob.policy(lp.cpu(), old.cpu(), adv.cpu(), ids, E, mean=mean)
    n = np.array([max(1, (ids == e).sum()) for e in range(E)])
    some = sum((ids == e).any() for e in range(E))
    w = 1 / (ids >= 0).sum() if mean == "token" else 1 / (n[np.maximum(ids, 0)] * some)
    terms = np.where(ids >= 0, w * 2.0 * np.abs(adv.double().cpu().numpy()), 0.0).sum()     # ratios below 2
    assert abs(out.loss.item() - want) <= 2.0 ** -19 * terms + 2.0 ** -81 + 2.0 ** -23 * abs(want)
    assert abs(out.stats[1].item() - share) <= 2.0 ** -23 * share


@pytest.mark.parametrize("kind", ["block", "warp", "lane", "token"])
@pytest.mark.parametrize("mean", ["token", "episode"])
@pytest.mark.parametrize("f", [1e-4, 1e-6, 3e-7, 1e-7, -1e-7, 1e-9, 1e-11])
def test_divergence_of_a_policy_that_has_just_started(pvl, kind, mean, f):
    """f^2 / 2 and more, all tokens the same: one rounding of f itself less."""
    ids, E = layout(kind)
    sid = torch.from_numpy(ids).cuda()
    ref = torch.full(ids.shape, f, device="cuda")
    out = pvl.pack_policy_fwd(torch.zeros_like(ref), None, torch.zeros_like(ref), sid, E, ref_logp=ref, kl_weight=1.0, mean=mean)
    x = float(ref[0])
    want = x * x / 2 + x ** 3 / 6 + x ** 4 / 24
    for got in (out.stats[0].item(), out.loss.item()):
        assert abs(got - want) <= 2.0 ** -20 * want + 2.0 ** -81, (got, want)


def test_small_terms_beside_large_ones(pvl):
    """Episodes of other sizes in one warp: each mean by itself."""
    ids = (torch.arange(4096, device="cuda", dtype=torch.int32) // 4) % 8
    size = torch.tensor([1.0, 1e-3, 1e-6, 1e-9, 1e-12, 1e-14, 2e3, 3e6], device="cuda")
    rewards = pvl.pack_preference_fwd(size[ids.long()].contiguous(), None, ids,
                                      torch.arange(8, dtype=torch.int32, device="cuda").view(4, 2), 8, beta=1.0, mean=True).rewards
    want = size.double().view(4, 2)
    assert ((rewards.double() - want).abs() <= 2.0 ** -22 * want + 2.0 ** -81).all()


@pytest.mark.parametrize("gap", [20.0, 35.0, 40.0, 45.0, 50.0])
def test_factors_of_pairs_won_by_far(pvl, gap):
    """beta sigmoid(-gap) for the chosen and the rejected alike: relative to four roundings of the gap and 2^-19 for exp
    and quotient."""
    ids = torch.arange(2, dtype=torch.int32, device="cuda").repeat_interleave(10)
    lp = torch.zeros(20, device="cuda")
    lp[0] = gap
    out = pvl.pack_preference_fwd(lp, None, ids, torch.tensor([[0, 1]], dtype=torch.int32, device="cuda"), 2, beta=1.0)
    want = math.exp(-gap) / (1 + math.exp(-gap))
    tol = 2.0 ** -22 * (8 + gap) * want + 2.0 ** -80
    assert abs(out.coef[0].item() + want) <= tol and abs(out.coef[1].item() - want) <= tol


@pytest.mark.parametrize("f", [3.0, 4.0, 8.0, 40.0, 84.0, 86.0, 88.0, 88.5])
def test_large_divergence(pvl, f):
    """Finite up to the largest fp32; exp carries 2^-22, and 2^-24 |f| for its argument."""
    ids = torch.full((9,), -1, dtype=torch.int32, device="cuda")
    ids[4] = 0
    ref = torch.full((9,), f, device="cuda")
    zero = torch.zeros_like(ref)
    out = pvl.pack_policy_fwd(zero, None, zero, ids, 1, ref_logp=ref, kl_weight=1.0)
    want = math.expm1(f) - f
    for got in (out.stats[0].item(), out.loss.item()):
        assert abs(got - want) <= 2.0 ** -19 * want, (got, want)


@pytest.mark.parametrize("mean", ["token", "episode"])
@pytest.mark.parametrize("ratio", ["token", "episode"])
@pytest.mark.parametrize("N,E", [(64, 1), (5000, 1), (5000, 40), (9000, 700)])
def test_means_of_large_terms(pvl, mean, ratio, N, E):
    """Sums past the largest fp32 whose means are not, of the divergence and of the loss, beside small ones."""
    ids = np.sort(np.arange(N) % E).astype(np.int32)
    sid = torch.from_numpy(ids).cuda()
    ref = torch.full((N,), 88.0, device="cuda")
    ref[::7] = 0.5
    zero = torch.zeros(N, device="cuda")
    small = torch.zeros(E, device="cuda")
    out = pvl.pack_policy_fwd(zero, zero, small, sid, E, ref_logp=ref, kl_weight=0.5, ratio=ratio, mean=mean)
    loss, kl, _, grad = ob.policy(zero.cpu(), zero.cpu(), small.cpu(), ids, E, ref_logp=ref.cpu(), kl_weight=0.5, ratio=ratio, mean=mean)
    assert math.isfinite(out.loss.item()) and abs(out.loss.item() - loss) <= 2.0 ** -19 * abs(loss)
    assert abs(out.stats[0].item() - kl) <= 2.0 ** -19 * kl
    d = pvl.pack_policy_bwd(None, zero, zero, small, sid, out.coef, ref_logp=ref, kl_weight=0.5, ratio=ratio)
    assert (np.abs(d.double().cpu().numpy() - grad) <= 2.0 ** -19 * np.abs(grad)).all()
    adv = torch.full((E,), -3e38, device="cuda")
    adv[1::3] = 1.0
    out = pvl.pack_policy_fwd(zero, zero, adv, sid, E, ratio=ratio, mean=mean)
    loss = ob.policy(zero.cpu(), zero.cpu(), adv.cpu(), ids, E, ratio=ratio, mean=mean)[0]
    assert abs(out.loss.item() - loss) <= 2.0 ** -19 * abs(loss)
    # infinities still are
    ref[3] = 200.0
    out = pvl.pack_policy_fwd(zero, zero, small, sid, E, ref_logp=ref, kl_weight=0.5, ratio=ratio, mean=mean)
    assert out.loss.item() == math.inf and out.stats[0].item() == math.inf


@pytest.mark.parametrize("kind", ["sigmoid", "hinge"])
def test_mean_of_pairs_lost_by_the_lowest_value(pvl, kind):
    """Forty pairs, each of a loss of 3.4e37: their sum leaves fp32, their mean does not."""
    ids = torch.arange(4, dtype=torch.int32, device="cuda").repeat_interleave(10)
    lp = torch.full((40,), -1.0, device="cuda")
    low = torch.finfo(torch.float32).min
    lp[3] = low
    pairs = torch.tensor([[0, 1]] * 40 + [[2, 3]] * 40, dtype=torch.int32, device="cuda")
    out = pvl.pack_preference_fwd(lp, None, ids, pairs, 4, kind=kind)
    assert out.loss.item() == pytest.approx(-0.1 * low / 2, rel=1e-6)
    own = 0.05 if kind == "sigmoid" else 0.1
    assert torch.allclose(out.coef.cpu(), torch.tensor([-0.1 / 2, 0.1 / 2, -own / 2, own / 2]), rtol=1e-6)
