"""The oracle's log-probabilities, preference and policy losses and AdamW step against library routines in fp64,
differences and closed forms (CPU only)."""

import math

import numpy as np
import pytest
import torch

from oracle import adamw, objectives as ob


def differences(f, x, at, h=1e-6):
    out = []
    for i in at:
        up, down = x.copy(), x.copy()
        up[i] += h
        down[i] -= h
        out.append((f(up) - f(down)) / (2 * h))
    return np.array(out)


@pytest.mark.parametrize("T", [1.0, 0.7])
def test_logprob_against_torch(T):
    g = torch.Generator().manual_seed(1)
    x = torch.randn(2, 5, 11, generator=g, dtype=torch.float64).requires_grad_()
    t = torch.randint(0, 11, (2, 5), generator=g)
    ids = torch.tensor([[0, 0, -1, 0, 0], [1, 1, 1, -1, -1]])
    up, ue = torch.randn(2, 5, generator=g, dtype=torch.float64), torch.randn(2, 5, generator=g, dtype=torch.float64)
    valid = ob.valid_targets(t, 11, ids)
    assert (valid == (ids >= 0).numpy()).all()
    logs = torch.log_softmax(x / T, 2)
    lp = logs.gather(2, t[..., None])[..., 0]
    ent = -(logs.exp() * logs).sum(2)
    mask = torch.from_numpy(valid).double()
    grad, = torch.autograd.grad(((lp * up + ent * ue) * mask).sum(), x)
    a, b, c = ob.logprob(x, t, valid, T)
    assert np.allclose(a, (lp * mask).detach(), atol=1e-13) and np.allclose(c, (ent * mask).detach(), atol=1e-13)
    assert np.allclose(b, (torch.logsumexp(x / T, 2) * mask).detach(), atol=1e-13)
    assert np.allclose(ob.logprob_grad(x, t, valid, up, ue, T), grad, atol=1e-13)


def test_logprob_targets_outside_and_banned_logits():
    x = np.zeros((1, 4, 3))
    x[0, :, 2] = -np.inf
    t = np.array([[0, -100, 3, 2]])
    valid = ob.valid_targets(t, 3)
    assert valid.tolist() == [[True, False, False, True]]
    lp, lse, ent = ob.logprob(x, t, valid)
    assert np.allclose(lp[0, :3], [-math.log(2), 0, 0]) and lp[0, 3] == -np.inf
    assert np.allclose(lse[0], [math.log(2), 0, 0, math.log(2)]) and np.allclose(ent[0, 0], math.log(2))
    g = ob.logprob_grad(x, t, valid, np.ones((1, 4)), np.ones((1, 4)))
    assert np.isfinite(g).all() and np.allclose(g[0, 0], [0.5, -0.5, 0]) and not g[0, 1:3].any()


IDS = np.array([[0, 0, 0, -1, 1, 1, -1], [2, 2, 3, 3, 3, 3, -1]])


@pytest.mark.parametrize("kind", ["sigmoid", "squared", "hinge"])
@pytest.mark.parametrize("mean", [False, True])
def test_preference_gradient(kind, mean):
    rng = np.random.default_rng(2)
    lp, ref = rng.normal(size=IDS.shape), rng.normal(size=IDS.shape)
    pairs = np.array([[0, 1], [2, 3], [0, 3], [-1, 2], [1, 1]])
    how = dict(beta=0.6, kind=kind, smoothing=0.1 if kind == "sigmoid" else 0.0, margin=0.2, mean=mean)
    loss, rewards, coef, grad = ob.preference(lp, ref, IDS, pairs, 5, **how)
    at = [tuple(i) for i in np.ndindex(IDS.shape)]
    assert np.allclose(differences(lambda x: ob.preference(x, ref, IDS, pairs, 5, **how)[0], lp, at), grad.reshape(-1), atol=1e-8)
    assert not rewards[3].any() and coef[4] == 0.0 and not grad[IDS < 0].any()
    if kind == "sigmoid" and not mean:
        D = [np.sum((lp - ref)[IDS == e]) for e in range(4)]
        x = [0.6 * (D[c] - D[r] - 0.2) for c, r in ((0, 1), (2, 3), (0, 3), (1, 1))]
        ls = torch.nn.functional.logsigmoid(torch.tensor(x)), torch.nn.functional.logsigmoid(-torch.tensor(x))
        assert np.isclose(loss, float(-(0.9 * ls[0] + 0.1 * ls[1]).mean()))


@pytest.mark.parametrize("ratio", ["token", "episode"])
@pytest.mark.parametrize("mean", ["token", "episode"])
def test_policy_gradient(ratio, mean):
    rng = np.random.default_rng(3)
    lp = rng.normal(size=IDS.shape)
    old, ref = lp + 0.3 * rng.normal(size=IDS.shape), lp + 0.5 * rng.normal(size=IDS.shape)
    adv = rng.normal(size=5) if ratio == "episode" else rng.normal(size=IDS.shape)
    how = dict(ref_logp=ref, clip_low=0.1, clip_high=0.15, kl_weight=0.3, ratio=ratio, mean=mean)
    loss, kl, share, grad = ob.policy(lp, old, adv, IDS, 5, **how)
    at = [tuple(i) for i in np.ndindex(IDS.shape)]
    assert np.allclose(differences(lambda x: ob.policy(x, old, adv, IDS, 5, **how)[0], lp, at), grad.reshape(-1), atol=1e-8)
    assert 0 < share < 1 and kl > 0 and not grad[IDS < 0].any()
    # token by token: min of the two products
    r = np.exp(lp - old)
    if ratio == "token" and mean == "token":
        pg = -np.minimum(r * adv, np.clip(r, 0.9, 1.15) * adv)
        f = ref - lp
        ok = IDS >= 0
        assert np.isclose(loss, (pg + 0.3 * (np.exp(f) - f - 1))[ok].mean())
        # without an old policy and a divergence: minus the mean advantage
        assert np.isclose(ob.policy(lp, None, adv, IDS, 5)[0], -adv[ok].mean())


def test_no_tokens_and_no_pairs():
    none = np.full((1, 4), -1)
    lp = np.zeros((1, 4))
    assert ob.preference(lp, None, none, np.array([[0, 1]]), 2)[0] == pytest.approx(math.log(2))
    assert ob.preference(lp, None, none, np.array([[-1, -1]]), 2)[0] == 0.0
    loss, kl, share, grad = ob.policy(lp, lp, np.zeros(2), none, 2, ratio="episode", mean="episode")
    assert (loss, kl, share) == (0.0, 0.0, 0.0) and not grad.any()


def test_adamw_against_torch():
    g = torch.Generator().manual_seed(4)
    p = torch.randn(40, generator=g, dtype=torch.float64)
    ours, m, v = p.numpy().copy(), np.zeros(40), np.zeros(40)
    q = p.clone().requires_grad_()
    opt = torch.optim.AdamW([q], lr=1e-2, betas=(0.8, 0.95), eps=1e-6, weight_decay=0.1)
    for t in range(1, 6):
        grad = torch.randn(40, generator=g, dtype=torch.float64)
        q.grad = grad
        opt.step()
        ours, m, v, _ = adamw.step(ours, grad.numpy(), m, v, t, 1e-2, (0.8, 0.95), 1e-6, 0.1)
        assert np.allclose(ours, q.detach(), atol=1e-13)


def test_eight_bits():
    """Codes are e4m3 values next to what they stand for; chances are spread evenly."""
    rng = np.random.default_rng(5)
    x = rng.normal(size=(64, 256)) * 10.0 ** rng.uniform(-4, 4, size=(64, 1))
    x[:, 7] *= 1e-9
    um, uv = adamw.chances(np.arange(64), 3, 11)
    for u, positive in ((um, False), (uv, True)):
        y = np.abs(x) if positive else x
        code, scale, near = adamw.encode(y, u, positive)
        as_float = torch.from_numpy(code).to(torch.float8_e4m3fn).double().numpy()
        assert (as_float == code).all() and (np.abs(code).max(1) == 448).all()
        exact = y / scale[:, None]
        assert (np.abs(code - exact) <= adamw.e4m3_step(exact) * (1 + 1e-12)).all()
        assert (near >= 0).all() and (near <= 0.5).all()
        assert ((code != 0).all() if positive else True)
    u = np.concatenate([um.ravel(), uv.ravel()])
    # 32768 values: the mean of as many even draws has a deviation of 0.2887 / sqrt(32768) = 0.0016
    assert abs(u.mean() - 0.5) < 6 * 0.0016 and 0 < u.min() and u.max() < 1
    assert abs(np.corrcoef(um.ravel(), uv.ravel())[0, 1]) < 6 / math.sqrt(um.size)
    again = adamw.chances(np.arange(64), 4, 11)[0]
    assert abs(np.corrcoef(um.ravel(), again.ravel())[0, 1]) < 6 / math.sqrt(um.size)
