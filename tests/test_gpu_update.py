"""Log-probabilities, losses over packed episodes, norm and update as they are used: one after the other behind packed
attention, through autograd, on other streams, captured and replayed, and what they refuse (GPU)."""

import math

import numpy as np
import pytest
import torch

from oracle import adamw as oa

pytestmark = pytest.mark.gpu

LAYOUT = dict(frames=[[5, 3, 6]], valid=[[5, 2, 6]], tokens=16, L=256, E=3)


@pytest.fixture(scope="module")
def pvl(cuda_ok):
    import packed_variable_length_gb300 as p
    return p


def to_np(t):
    return t.detach().double().cpu().numpy()


def randn(*shape, seed, dtype=torch.float32, mul=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(*shape, generator=g) * mul).to(dtype).cuda()


def plain_policy(logp, old, ref, adv, ids, low, high, klw):
    ok = ids >= 0
    d = (logp - old)[ok]
    a = adv[ids[ok].long()]
    pg = -torch.minimum(d.exp() * a, d.exp().clamp(1 - low, 1 + high) * a)
    f = (ref - logp)[ok]
    return (pg + klw * (f.exp() - f - 1)).mean()


@pytest.mark.parametrize("bits", [32, 8])
def test_training_steps_behind_attention(pvl, bits):
    """Attention over a pack, a head, log-probabilities, the policy loss with an entropy bonus, backward, norm, update;
    three steps.  The logits' gradient against fp64 from the same logits: rounded once to bf16 (2^-8), and before that
    2^-16 of the probability's and the target's part; parameters against the oracle's step from their own gradients."""
    H, D, V = 2, 64, 301
    sid = pvl.pack_build_seq_ids(LAYOUT["frames"], LAYOUT["valid"], LAYOUT["tokens"], LAYOUT["L"])
    L, E = LAYOUT["L"], LAYOUT["E"]
    x = randn(1, L, H * D, seed=1, dtype=torch.bfloat16)
    params = [randn(3 * H * D, H * D, seed=2, mul=0.1), randn(V, H * D, seed=3, mul=0.2), randn(V, seed=4, mul=0.1)]
    params = [p.bfloat16().requires_grad_() for p in params]
    state = pvl.adamw_state(params, bits=bits, seed=3)
    targets = torch.randint(0, V, (1, L), generator=torch.Generator().manual_seed(5)).cuda()
    adv = torch.tensor([1.0, -0.5, 2.0], device="cuda")
    old = ref = None
    losses = []
    for step in range(3):
        q, k, v = (x @ params[0].t()).view(1, L, 3, H, D).unbind(2)
        o = pvl.packed_attention(q.contiguous(), k.contiguous(), v.contiguous(), sid)
        logits = o.flatten(2) @ params[1].t() + params[2]
        logits.retain_grad()
        logp, ent = pvl.token_logprob(logits, targets, sid, temperature=0.9, entropy=True)
        if old is None:
            old, ref = logp.detach() + randn(1, L, seed=6, mul=0.1), logp.detach() + randn(1, L, seed=7, mul=0.2)
        loss, stats = pvl.policy_loss(logp, old, adv, sid, E, ref_logp=ref, kl_weight=0.1)
        assert not stats.requires_grad
        (loss - 0.01 * ent.sum() / L).backward()
        pvl.device_error()
        # the same from the logits in 64 bits
        z = logits.detach().double().requires_grad_()
        logs = torch.log_softmax(z / 0.9, 2)
        ok = sid >= 0
        lp = logs.gather(2, targets[..., None])[..., 0]
        en = -(logs.exp() * logs).sum(2)
        plain = plain_policy(lp, old.double(), ref.double(), adv.double(), sid, 0.2, 0.2, 0.1)
        up, ue = torch.autograd.grad(plain, lp, retain_graph=True)[0], 0.01 / L
        (plain - 0.01 * en[ok].sum() / L).backward()
        assert abs(loss.item() - plain.item()) < 2.0 ** -18 * (1 + abs(plain.item()))
        got, want = logits.grad.double(), z.grad
        assert not got[~ok].any()
        prob = logs.detach().exp()
        slack = 2.0 ** -16 * (prob * (up.abs()[..., None] + ue * (logs.detach().abs() + en.detach()[..., None] + 2)) / 0.9)
        slack = slack.scatter_add(2, targets[..., None], 2.0 ** -16 * up.abs()[..., None] / 0.9)
        assert (((got - want).abs() <= 2.0 ** -8 * want.abs() + slack)[ok]).all()
        losses.append(loss.item())
        # norm and update
        grads = [p.grad for p in params]
        norm = pvl.grad_norm(grads)
        size = oa.grad_norm([to_np(g) for g in grads])
        assert abs(norm.item() - size) <= 2.0 ** -18 * size
        before = [to_np(state.masters(i)) for i in range(3)]
        moments = [tuple(map(to_np, state.moments(i))) for i in range(3)]
        pvl.adamw_step(params, grads, state, 1e-2, weight_decay=[0.1, 0.1, 0.0], grad_norm=norm, max_norm=0.5)
        for i, (p, g) in enumerate(zip(params, grads)):
            want, m, v2, change = oa.step(before[i], to_np(g), *moments[i], step + 1, 1e-2, decay=[0.1, 0.1, 0.0][i],
                                          clip=min(1.0, 0.5 / norm.item()))
            size = 0.9 * np.abs(moments[i][0]) + 0.1 * np.abs(to_np(g))
            part = 1e-2 / (1 - 0.9 ** (step + 1)) * 2.0 ** -21 * size / (np.sqrt(v2 / (1 - 0.999 ** (step + 1))) + 1e-8)
            assert (np.abs(to_np(state.masters(i)) - want) <= 2.0 ** -22 * np.abs(before[i]) + 2.0 ** -19 * np.abs(change) + part).all()
            assert torch.equal(p, state.masters(i).bfloat16())
            p.grad = None
    assert len(set(losses)) == 3 and state.steps.tolist() == [3, 3, 3]


@pytest.mark.parametrize("kind", ["sigmoid", "squared", "hinge"])
def test_preference_through_autograd(pvl, kind):
    """Logits to the loss over pairs: along random directions, the gradient against differences.  A loss is good to
    2^-20 (1 + |loss|), so a difference over 2 h is to 2^-20 (1 + |loss|) / h; a direction of length 1 changes logits by
    at most h, whose third-order part is below 4 h^2."""
    V, h = 97, 2.0 ** -6
    sid = pvl.pack_build_seq_ids(LAYOUT["frames"], LAYOUT["valid"], LAYOUT["tokens"], LAYOUT["L"])
    x = randn(1, LAYOUT["L"], V, seed=11).requires_grad_()
    ref = randn(1, LAYOUT["L"], seed=12) - 5.0
    t = torch.randint(0, V, (1, LAYOUT["L"]), generator=torch.Generator().manual_seed(13), dtype=torch.int32).cuda()
    pairs = torch.tensor([[0, 1], [2, 1], [0, 2]], dtype=torch.int32, device="cuda")

    def loss_of(x):
        logp = pvl.token_logprob(x, t, sid)
        return pvl.preference_loss(logp, ref, sid, pairs, LAYOUT["E"], beta=0.5, kind=kind, mean=True)

    loss, rewards = loss_of(x)
    assert rewards.shape == (3, 2) and not rewards.requires_grad
    (3.0 * loss).backward()
    assert not x.grad[(sid < 0)].any()
    for seed in range(20, 24):
        d = randn(*x.shape, seed=seed)
        d = d / d.norm()
        with torch.no_grad():
            slope = (loss_of(x + h * d)[0] - loss_of(x - h * d)[0]).item() / (2 * h)
        assert abs(3 * slope - (x.grad * d).sum().item()) <= 3 * (2.0 ** -20 * (1 + abs(loss.item())) / h + 4 * h * h) * 1.01


def test_gradients_of_parts_and_orders(pvl):
    """The gradient of the entropy alone, of one output used twice, of none; a second derivative is refused."""
    x = randn(2, 5, 33, seed=31).requires_grad_()
    t = torch.zeros(2, 5, dtype=torch.int32, device="cuda")
    logp, ent = pvl.token_logprob(x, t, entropy=True)
    z = x.detach().double().requires_grad_()
    logs = torch.log_softmax(z, 2)
    for outs, plain in ((ent.sum(), -(logs.exp() * logs).sum()), ((logp * logp).sum(), (logs[..., 0] ** 2).sum())):
        g, = torch.autograd.grad(outs, x, retain_graph=True)
        w, = torch.autograd.grad(plain, z, retain_graph=True)
        assert torch.allclose(g.double(), w, rtol=2.0 ** -16, atol=2.0 ** -16)
    # a gradient that is broadcast, and one that comes transposed
    g, = torch.autograd.grad(logp, x, torch.ones(5, 2, device="cuda").t() * 2.0, retain_graph=True)
    w, = torch.autograd.grad(2.0 * logp.sum(), x, retain_graph=True)
    assert torch.equal(g, w)
    g, = torch.autograd.grad(logp.sum(), x, create_graph=True)
    with pytest.raises(RuntimeError):
        g.sum().backward()
    lp = logp.detach().requires_grad_()
    sid = torch.zeros(2, 5, dtype=torch.int32, device="cuda")
    loss, _ = pvl.policy_loss(lp, lp.detach() - 0.1, torch.ones(1, device="cuda"), sid, 1)
    g, = torch.autograd.grad(loss, lp, create_graph=True)
    with pytest.raises(RuntimeError):
        g.sum().backward()


def test_a_graph_older_than_the_update_is_refused(pvl):
    """The update counts as a change in place, as autograd has it for its own."""
    w = randn(8, 8, seed=41).requires_grad_()
    y = (w * w).sum()
    state = pvl.adamw_state([w])
    pvl.adamw_step([w], [torch.ones_like(w)], state, 1e-2)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        y.backward()


def everything(pvl, st, stream=None):
    """One pass of all entry points on a stream; what they give."""
    s = dict(stream=stream)
    logp, lse, ent = pvl.pack_logprob_fwd(st["x"], st["t"], st["ids"], entropy=True, **s)
    pref = pvl.pack_preference_fwd(logp, st["ref"], st["ids"], st["pairs"], 3, **s)
    d1 = pvl.pack_preference_bwd(None, pref.coef, st["ids"], **s)
    pol = pvl.pack_policy_fwd(logp, st["old"], st["adv"], st["ids"], 3, ref_logp=st["ref"], kl_weight=0.1, **s)
    d2 = pvl.pack_policy_bwd(None, logp, st["old"], st["adv"], st["ids"], pol.coef, ref_logp=st["ref"], kl_weight=0.1, **s)
    dx = pvl.pack_logprob_bwd(d2, st["x"], st["t"], lse, st["ids"], ent=ent, dent=d1, **s)
    norm = pvl.grad_norm([dx], **s)
    pvl.adamw_step([st["w"]], [dx], st["state"], st["lr"], grad_norm=norm, max_norm=0.01, **s)
    return [logp, lse, ent, *pref, d1, *pol, d2, dx, norm]


def inputs(pvl, seed=51, V=513):
    L = LAYOUT["L"]
    st = {"x": randn(1, L, V, seed=seed, mul=2.0), "old": randn(1, L, seed=seed + 1) - 6, "ref": randn(1, L, seed=seed + 2) - 6,
          "adv": randn(3, seed=seed + 3), "w": randn(1, L, V, seed=seed + 4)}
    st["ids"] = pvl.pack_build_seq_ids(LAYOUT["frames"], LAYOUT["valid"], LAYOUT["tokens"], L)
    st["t"] = torch.randint(0, V, (1, L), generator=torch.Generator().manual_seed(seed), dtype=torch.int32).cuda()
    st["pairs"] = torch.tensor([[0, 1], [2, 0]], dtype=torch.int32, device="cuda")
    st["state"] = pvl.adamw_state([st["w"]], bits=8, seed=1)
    st["lr"] = torch.tensor([1e-2], device="cuda")
    return st


def outcome(st, outs):
    torch.cuda.synchronize()
    return [t.clone() for t in (*outs, st["w"], st["state"].m.view(torch.uint8), st["state"].v.view(torch.uint8),
                                st["state"].m_scale, st["state"].steps)]


def test_other_streams(pvl):
    """A stream passed, a stream made current, and two streams at once, all with the same bits as the default one."""
    st = inputs(pvl)
    want = outcome(st, everything(pvl, st))
    side = torch.cuda.Stream()
    for how in ("passed", "current", "handle"):
        st = inputs(pvl)
        side.wait_stream(torch.cuda.current_stream())
        if how == "current":
            with torch.cuda.stream(side):
                outs = everything(pvl, st)
        else:
            outs = everything(pvl, st, stream=side if how == "passed" else side.cuda_stream)
        assert all(torch.equal(a, b) for a, b in zip(want, outcome(st, outs))), how
    pair = [inputs(pvl), inputs(pvl)]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    got = [None, None]
    for _ in range(3):
        for i in (0, 1):
            with torch.cuda.stream(streams[i]):
                got[i] = everything(pvl, pair[i])
    torch.cuda.synchronize()
    for a, b in zip(got[0], got[1]):
        assert torch.equal(a, b)
    assert torch.equal(pair[0]["w"], pair[1]["w"]) and pair[0]["state"].steps.item() == 3


def test_captured_and_replayed(pvl):
    """The whole pass captured once; replays step as eager calls do, with the rate read from the device."""
    eager = inputs(pvl)
    want = []
    for i in range(3):
        eager["lr"].fill_(1e-2 / (i + 1))
        want.append(outcome(eager, everything(pvl, eager)))
    st = inputs(pvl)
    warm = inputs(pvl, seed=90)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        everything(pvl, warm)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = everything(pvl, st)
    for i in range(3):
        st["lr"].fill_(1e-2 / (i + 1))
        graph.replay()
        assert all(torch.equal(a, b) for a, b in zip(want[i], outcome(st, outs))), i


def test_autograd_captured_and_replayed(pvl):
    """Forward and backward through autograd in one captured graph, replayed on other logits; no eager graph of the
    leaves lives while it is captured."""
    L, E = LAYOUT["L"], LAYOUT["E"]
    sid = pvl.pack_build_seq_ids(LAYOUT["frames"], LAYOUT["valid"], LAYOUT["tokens"], L)
    t = torch.randint(0, 65, (1, L), generator=torch.Generator().manual_seed(1)).cuda()
    old, adv = randn(1, L, seed=71) * 0.1 - 4.2, randn(E, seed=72)
    pairs = torch.tensor([[0, 1], [2, 1]], dtype=torch.int32, device="cuda")
    x = randn(1, L, 65, seed=73).requires_grad_()

    def step():
        logp, ent = pvl.token_logprob(x, t, sid, entropy=True)
        a, _ = pvl.policy_loss(logp, old, adv, sid, E, mean="episode")
        b, _ = pvl.preference_loss(logp, old, sid, pairs, E, mean=True)
        loss = a + b - 0.01 * ent.mean()
        return loss.detach(), torch.autograd.grad(loss, x)[0]

    fresh = [randn(1, L, 65, seed=80 + i) for i in range(3)]
    want = []
    for v in fresh:
        with torch.no_grad():
            x.copy_(v)
        want.append([r.clone() for r in step()])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = step()
    for i in (2, 0, 1):
        with torch.no_grad():
            x.copy_(fresh[i])
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(outs, want[i])), i


def test_graphs_that_share_a_workspace(pvl):
    """Two captured calls of other sizes with one workspace, replayed in turn: what it holds on entry does not matter."""
    ws = torch.full((max(pvl.pack_policy_ws_bytes(40), pvl.pack_preference_ws_bytes(40)),), 0xAB, dtype=torch.uint8, device="cuda")
    st = inputs(pvl)
    lp = randn(1, LAYOUT["L"], seed=61)
    wide = torch.arange(5000, device="cuda", dtype=torch.int32).view(1, -1) % 40
    lw, adv = randn(1, 5000, seed=62), randn(40, seed=63)
    calls = [lambda: pvl.pack_policy_fwd(lp, lp - 0.1, st["adv"], st["ids"], 3, mean="episode", ws=ws),
             lambda: pvl.pack_policy_fwd(lw, lw + 0.1, adv, wide, 40, ratio="episode", ws=ws),
             lambda: pvl.pack_preference_fwd(lw, None, wide, st["pairs"], 40, ws=ws)]
    want = [[t.clone() for t in c()] for c in calls]
    graphs, outs = [], []
    for c in calls:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(c())
        graphs.append(g)
    for i in (0, 1, 2, 1, 0, 2, 2, 1):
        for t in outs[i]:
            t.zero_()
        graphs[i].replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(outs[i], want[i])), i


def test_refusals(pvl):
    """Tensors of another type, shape or device, or with gaps, and lists that do not belong to their state."""
    st = inputs(pvl)
    x, t, ids, old, adv = st["x"], st["t"], st["ids"], st["old"], st["adv"]
    lp, lse, ent = pvl.pack_logprob_fwd(x, t, ids, entropy=True)
    two = torch.zeros(1, 2 * LAYOUT["L"], device="cuda")[:, ::2]
    bad_rows = (lp[:, 1:], lp.double(), lp.cpu(), two, lp[0])
    for bad in (t[:, 1:], t.cpu(), t.float(), torch.zeros(1, 2 * LAYOUT["L"], dtype=torch.int32, device="cuda")[:, ::2]):
        with pytest.raises(ValueError):
            pvl.pack_logprob_fwd(x, bad)
        with pytest.raises(ValueError):
            pvl.pack_logprob_fwd(x, t, bad)
    with pytest.raises(ValueError):
        pvl.pack_logprob_fwd(x.transpose(1, 2), t)
    with pytest.raises(ValueError):
        pvl.pack_logprob_fwd(x.half(), t)
    with pytest.raises(pvl.PvlError):
        pvl.pack_logprob_fwd(x, t, temperature=0.0)
    for bad in bad_rows:
        for call in (lambda: pvl.pack_logprob_fwd(x, t, logp=bad), lambda: pvl.pack_logprob_fwd(x, t, lse=bad),
                     lambda: pvl.pack_logprob_bwd(bad, x, t, lse), lambda: pvl.pack_logprob_bwd(lp, x, t, bad),
                     lambda: pvl.pack_logprob_bwd(lp, x, t, lse, ent=ent, dent=bad),
                     lambda: pvl.pack_preference_fwd(bad, None, ids, st["pairs"], 3),
                     lambda: pvl.pack_preference_fwd(lp, bad, ids, st["pairs"], 3),
                     lambda: pvl.pack_policy_fwd(bad, old, adv, ids, 3), lambda: pvl.pack_policy_fwd(lp, bad, adv, ids, 3),
                     lambda: pvl.pack_policy_fwd(lp, old, bad, ids, 3), lambda: pvl.pack_policy_fwd(lp, old, adv, ids, 3, ref_logp=bad)):
            with pytest.raises(ValueError):
                call()
    for bad in (x.bfloat16(), x[:, 1:], x.cpu(), x[..., :-1]):
        with pytest.raises(ValueError):
            pvl.pack_logprob_bwd(lp, x, t, lse, dlogits=bad)
    with pytest.raises(pvl.PvlError, match="overlap"):
        pvl.pack_logprob_bwd(lp, x, t, lse, dlogits=torch.zeros(x.shape[2], device="cuda").expand(x.shape))
    for pairs in (st["pairs"].long(), st["pairs"][:, :1], st["pairs"].cpu(), st["pairs"].t()):
        with pytest.raises(ValueError):
            pvl.pack_preference_fwd(lp, None, ids, pairs, 3)
    for kw in (dict(kind="other"), dict(ws=torch.zeros(4, device="cuda"))):
        with pytest.raises(ValueError):
            pvl.pack_preference_fwd(lp, None, ids, st["pairs"], 3, **kw)
    for kw in (dict(beta=0.0), dict(smoothing=0.7), dict(kind="hinge", smoothing=0.1), dict(margin=math.inf),
               dict(ws=torch.zeros(16, dtype=torch.uint8, device="cuda"))):
        with pytest.raises(pvl.PvlError):
            pvl.pack_preference_fwd(lp, None, ids, st["pairs"], 3, **kw)
    with pytest.raises(pvl.PvlError):
        pvl.pack_preference_fwd(lp, None, ids, st["pairs"][:0], 3)
    with pytest.raises(pvl.PvlError):
        pvl.pack_preference_fwd(lp, None, ids, st["pairs"], 0)
    for kw in (dict(ratio="batch"), dict(mean="batch")):
        with pytest.raises(ValueError):
            pvl.pack_policy_fwd(lp, old, adv, ids, 3, **kw)
    with pytest.raises(ValueError):
        pvl.pack_policy_fwd(lp, old, lp, ids, 3, ratio="episode")        # ratios of episodes, advantages of tokens
    for kw in (dict(clip_low=1.0), dict(clip_high=-0.1), dict(kl_weight=0.1), dict(kl_weight=-1.0, ref_logp=old)):
        with pytest.raises(pvl.PvlError):
            pvl.pack_policy_fwd(lp, old, adv, ids, 3, **kw)
    # the update
    w, state = st["w"], st["state"]
    other = [torch.zeros_like(w), torch.zeros(5, device="cuda")]
    pair = pvl.adamw_state(other)
    g = [torch.ones_like(p) for p in other]
    for params, grads in ((other[:1], g), (other, g[:1]), (other[::-1], g), (other, g[::-1]), ([other[0].bfloat16(), other[1]], g),
                          (other, [g[0].bfloat16(), g[1]]), (other, [g[0].half(), g[1].half()]), (other, [g[0], g[1].cpu()]),
                          (other, [g[0].transpose(1, 2).contiguous().transpose(1, 2), g[1]]), ([other[0].cpu(), other[1]], g)):
        with pytest.raises(ValueError):
            pvl.adamw_step(params, grads, pair, 1e-3)
    with pytest.raises(ValueError, match="twice"):
        pvl.adamw_state([w, w])
    same = [torch.zeros(4, device="cuda"), torch.zeros(4, device="cuda")]
    with pytest.raises(ValueError, match="twice"):
        pvl.adamw_step([same[0], same[0]], same, pvl.adamw_state(same), 1e-3)
    for kw in (dict(lr=torch.ones(2, device="cuda")), dict(lr=torch.ones(1)), dict(lr=torch.ones(1, device="cuda").double()),
               dict(max_norm=1.0), dict(grad_norm=torch.ones(2, device="cuda")), dict(weight_decay=[0.1]), dict(betas=None)):
        with pytest.raises(ValueError):
            pvl.adamw_step(other, g, pair, **{"lr": 1e-3, **kw})
    for kw in (dict(lr=math.nan), dict(betas=(1.0, 0.9)), dict(eps=0.0), dict(weight_decay=math.inf),
               dict(grad_norm=torch.ones(1, device="cuda"), max_norm=0.0)):
        with pytest.raises(pvl.PvlError):
            pvl.adamw_step(other, g, pair, **{"lr": 1e-3, **kw})
    for name in ("m", "v", "steps", "done"):
        kept = getattr(pair, name)
        setattr(pair, name, kept[:-1])
        with pytest.raises(ValueError):
            pvl.adamw_step(other, g, pair, 1e-3)
        setattr(pair, name, kept)
    for grads in ([g[0], g[1].bfloat16()], [g[0].transpose(1, 2)], [g[0].half()]):
        with pytest.raises(ValueError):
            pvl.grad_norm(grads)
    torch.cuda.synchronize()
    assert not other[0].any() and pair.steps.tolist() == [0, 0]
