"""Workloads of the end of a packed training step: log-probabilities of the
tokens from the logits, preference and clipped policy losses over packed
episodes, and the AdamW update with the norm of the gradients it clips by.

Sizes: the 64k pack, the padded batch of four rows of 10,944 tokens and its
ragged neighbours of 4,560 are the attention workloads' own, widths of 1536
the model's (12 heads of 128); vocabularies and group sizes are generic.
"""

import math

import numpy as np
import torch

own = False

BLOCK = 256           # elements that share a scale of the 8-bit states
TOP = 448.0           # largest e4m3 value
BETAS, EPS, LR, DECAY = (0.9, 0.999), 1e-8, 3e-5, 0.01


# ------------------------------------------------------------------- cases
def _logprob(name, **kw):
    base = {"op": "logprob", "dir": "fwd", "B": 1, "L": 1, "V": 256, "dtype": "bf16", "T": 1.0, "entropy": False,
            "banned": 0, "pad": 0.0}
    return {"name": name, **base, **kw}


def _preference(name, **kw):
    base = {"op": "preference", "B": 1, "L": 1, "K": 1, "P": 1, "kind": "sigmoid", "beta": 0.1, "smoothing": 0.0,
            "margin": 0.0, "mean": False}
    return {"name": name, **base, **kw}


def _policy(name, **kw):
    base = {"op": "policy", "B": 1, "L": 1, "K": 1, "ratio": "token", "mean": "token", "adv": "token", "ref": True,
            "low": 0.2, "high": 0.2, "kl": 0.05}
    return {"name": name, **base, **kw}


def _adamw(name, **kw):
    base = {"op": "adamw", "layers": 1, "width": 1536, "out": 192, "param": "fp32", "grad": "fp32", "bits": 32,
            "clip": False, "step": 1000}
    return {"name": name, **base, **kw}


def listed():
    return [
        # the actions sampled for eight episodes: one token each over a large vocabulary, latency only
        _logprob("logprob_token", B=8, V=128001),
        # a training step on the 64k pack
        _logprob("logprob_fwd_64k", L=65536, V=32768),
        _logprob("logprob_bwd_64k", dir="bwd", L=65536, V=32768),
        # fp32 logits of an odd, partly banned vocabulary, with temperature and entropy bonus, padded rows
        _logprob("logprob_bwd_ragged", dir="bwd", B=4, L=2281, V=50001, dtype="fp32", T=0.7, entropy=True, banned=61,
                 pad=0.3),
        # binned actions of the padded batch: many short rows
        _logprob("logprob_fwd_bins", B=4, L=10944, V=256, entropy=True, pad=0.2),
        # two pairs of the four padded episodes
        _preference("preference_padded", B=4, L=10944, K=1, P=2),
        # many short episodes, each in several pairs, means over their tokens
        _preference("preference_many", B=8, L=32768, K=64, P=2048, mean=True, margin=0.05, beta=2.0, smoothing=0.1),
        # token ratios with advantages of tokens on the 64k pack of seven episodes
        _policy("policy_pack64k", L=65536, K=7),
        # groups of answers, one reward each: ratios and means of whole episodes
        _policy("policy_groups", B=64, L=4096, K=8, ratio="episode", mean="episode", adv="episode", low=0.003, high=0.004),
        # one block of the model, fp32 throughout
        _adamw("adamw_block"),
        # 24 blocks, bf16 parameters over fp32 masters, clipped
        _adamw("adamw_model", layers=24, param="bf16", grad="bf16", clip=True),
        # the same with states of 8 bits
        _adamw("adamw_model_8bit", layers=24, param="bf16", grad="bf16", bits=8, clip=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["logprob", "logprob", "preference", "policy", "adamw", "adamw"])
    if op == "logprob":
        V = _log(rng, 2, 200000)
        dtype = rng.choice(["bf16", "bf16", "fp32"])
        N = min(_log(rng, 1, 65536), 1500000000 // V)
        B = min(_log(rng, 1, 16), N)
        return {"op": op, "dir": rng.choice(["fwd", "bwd"]), "B": B, "L": max(1, N // B), "V": V, "dtype": dtype,
                "T": rng.choice([1.0, 1.0, 0.7, 1.3]), "entropy": rng.random() < 0.5,
                "banned": rng.choice([0, min(V // 2, 61)]), "pad": rng.choice([0.0, 0.3])}
    if op == "preference":
        B, K = _log(rng, 1, 64), _log(rng, 2, 64)
        L = max(2 * K, _log(rng, 64, 1 << 20) // B)
        return {"op": op, "B": B, "L": L, "K": K, "P": _log(rng, 1, 4 * B * K),
                "kind": rng.choice(["sigmoid", "sigmoid", "squared", "hinge"]), "beta": rng.choice([0.05, 0.1, 0.5]),
                "smoothing": 0.0, "margin": rng.choice([0.0, 0.2]), "mean": rng.random() < 0.5}
    if op == "policy":
        B, K = _log(rng, 1, 64), _log(rng, 1, 64)
        L = max(2 * K, _log(rng, 64, 1 << 20) // B)
        ratio = rng.choice(["token", "episode"])
        wide = 0.2 if ratio == "token" else 0.01
        return {"op": op, "B": B, "L": L, "K": K, "ratio": ratio, "mean": rng.choice(["token", "episode"]),
                "adv": "episode" if ratio == "episode" else rng.choice(["token", "episode"]),
                "ref": rng.random() < 0.7, "low": wide, "high": rng.choice([wide, 1.4 * wide]), "kl": rng.choice([0.01, 0.1])}
    width = _log(rng, 40, 2048)
    layers = max(1, min(_log(rng, 1, 24), 600000000 // (12 * width * width)))
    return {"op": op, "layers": layers, "width": width, "out": _log(rng, 1, 1000), "param": rng.choice(["fp32", "bf16"]),
            "grad": rng.choice(["fp32", "bf16"]), "bits": rng.choice([32, 8]), "clip": rng.random() < 0.5,
            "step": rng.choice([0, 3, 1000, 200000])}


# ------------------------------------------------------------------- inputs
def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _randn(g, *shape, dtype=torch.float32, mul=1.0, add=0.0):
    out = torch.empty(shape, dtype=dtype, device="cuda")
    flat = out.view(-1)
    for i in range(0, flat.numel(), 1 << 27):      # in pieces: the fp32 draw of a large tensor need not be whole
        part = flat[i:i + (1 << 27)]
        part.copy_(torch.randn(part.shape, generator=g, device="cuda").mul_(mul).add_(add))
    return out


def _episodes(case, seed):
    """int32 [B, L]: K episodes a row laid end to end, each with a prompt that is not trained on (-1), a tail of -1."""
    rng = np.random.default_rng(seed)
    B, L, K = case["B"], case["L"], case["K"]
    ids = np.full((B, L), -1, dtype=np.int32)
    for b in range(B):
        ends = np.sort(rng.integers(L // 2, L + 1, size=1) if K == 1 else rng.integers(0, L + 1, size=K))
        start = 0
        for k, end in enumerate(ends):
            prompt = int(rng.uniform(0.0, 0.3) * (end - start))
            ids[b, start + prompt:end] = b * K + k
            start = end
    return torch.from_numpy(ids).cuda()


def _shapes(case):
    """Parameter shapes of a stack of blocks: projections, a feed-forward of four widths, norms, modulation, a head."""
    w = case["width"]
    block = [(w, w)] * 4 + [(4 * w, w), (w, 4 * w)] + [(w,)] * 6 + [(4 * w,), (6, w)]
    return block * case["layers"] + [(case["out"], w), (case["out"],)]


def _places(case):
    """(elements, start in a buffer of whole 8-element groups, start in the states' whole blocks) of each tensor; totals."""
    sizes = [math.prod(s) for s in _shapes(case)]
    flat, at, places = 0, 0, []
    for n in sizes:
        places.append((n, flat, at))
        flat += -(-n // 8) * 8
        at += -(-n // BLOCK) * BLOCK
    return places, flat, at


def _valid(case, g):
    """seq_id [B, L] of padded rows: -1 past each row's length."""
    B, L = case["B"], case["L"]
    keep = 1.0 - case["pad"] * torch.rand(B, 1, generator=g, device="cuda")
    at = torch.arange(L, device="cuda")[None]
    row = torch.arange(B, device="cuda", dtype=torch.int32)[:, None].expand(B, L)
    return torch.where(at < keep * L, row, torch.full_like(row, -1)).contiguous()


def prepare(case, seed):
    g = _gen(seed)
    st = {"case": case}
    if case["op"] == "logprob":
        B, L, V = case["B"], case["L"], case["V"]
        x = _randn(g, B * L, V, dtype=torch.bfloat16 if case["dtype"] == "bf16" else torch.float32, mul=2.0)
        t = torch.randint(0, V - case["banned"], (B, L), generator=g, device="cuda")
        x.scatter_add_(1, t.view(-1, 1), torch.full((B * L, 1), 6.0, device="cuda").to(x.dtype))    # likely tokens
        if case["banned"]:
            x[:, V - case["banned"]:] = -math.inf
        st["x"], st["t"] = x.view(B, L, V), t.int()
        st["ids"] = _valid(case, g) if case["pad"] else None
        if case["dir"] == "bwd":
            st["dlogp"] = _randn(g, B, L)
            st["dent"] = _randn(g, B, L, mul=0.1) if case["entropy"] else None
            st["lse"], st["ent"] = _statistics(st["x"], case)
        return st
    if case["op"] in ("preference", "policy"):
        B, L, E = case["B"], case["L"], case["B"] * case["K"]
        st["ids"] = _episodes(case, seed)
        st["logp"] = -_randn(g, B, L).abs_().mul_(2.0)
        st["ref"] = st["logp"] + _randn(g, B, L, mul=0.2)
        if case["op"] == "preference":
            rng = np.random.default_rng(seed + 1)
            c = rng.integers(0, E, size=case["P"])
            r = (c + rng.integers(1, max(2, E), size=case["P"])) % E
            st["pairs"] = torch.from_numpy(np.stack([c, r], 1).astype(np.int32)).cuda()
            return st
        st["old"] = st["logp"] + _randn(g, B, L, mul=0.15)
        st["adv"] = _randn(g, B, L) if case["adv"] == "token" else _randn(g, E)
        st["ref"] = st["ref"] if case["ref"] else None
        return st
    return _prepare_adamw(st, case, g)


def _statistics(x, case):
    """lse and entropy [B, L] of the rows, as the forward gave them (fp32), a piece of rows at a time."""
    V = x.shape[2]
    rows = x.view(-1, V)
    lse, ent = (torch.empty(rows.shape[0], device="cuda") for _ in range(2))
    step = max(1, (1 << 27) // V)
    for i in range(0, rows.shape[0], step):
        z = rows[i:i + step].double() / case["T"]
        s = torch.logsumexp(z, 1, keepdim=True)
        p = (z - s).exp()
        lse[i:i + step] = s[:, 0].float()
        ent[i:i + step] = -torch.where(p > 0, p * (z - s), 0.0).sum(1).float()
    return lse.view(x.shape[:2]), ent.view(x.shape[:2])


def _prepare_adamw(st, case, g):
    places, flat, total = _places(case)
    shapes = _shapes(case)
    pt = torch.float32 if case["param"] == "fp32" else torch.bfloat16
    gt = torch.float32 if case["grad"] == "fp32" else torch.bfloat16
    at = torch.zeros(total, dtype=torch.bool, device="cuda")       # whether an element of the states is a parameter's
    for n, _, a in places:
        at[a:a + n] = True
    st["flat"] = _randn(g, flat, mul=0.02).to(pt)
    st["grads_flat"] = _randn(g, flat, dtype=gt, mul=1e-3)
    st["params"] = [st["flat"][f:f + n].view(s) for s, (n, f, _) in zip(shapes, places)]
    st["grads"] = [st["grads_flat"][f:f + n].view(s) for s, (n, f, _) in zip(shapes, places)]
    new = case["step"] == 0
    m = _randn(g, total, mul=0.0 if new else 3e-4).mul_(at)
    v = _randn(g, total, mul=0.0 if new else 1e-3).square_().mul_(at)
    buf = {"steps": torch.full((len(shapes),), case["step"], dtype=torch.int32, device="cuda")}
    if case["param"] == "bf16":
        buf["master"] = _randn(g, total, mul=0.02).mul_(at)
        for p, (n, _, a) in zip(st["params"], places):
            p.copy_(buf["master"][a:a + n].view(p.shape))
    if case["bits"] == 8:
        for key, t in (("m", m), ("v", v.sqrt_())):
            rows = t.view(-1, BLOCK)
            scale = rows.abs().amax(1) / TOP
            buf[key + "_scale"] = scale
            codes = rows / torch.where(scale > 0, scale, 1.0)[:, None]
            codes = torch.where((codes > 0) & (codes < 2.0 ** -9), 2.0 ** -9, codes) if key == "v" else codes
            buf[key] = codes.view(-1).to(torch.float8_e4m3fn)
    else:
        buf["m"], buf["v"] = m, v
    st["buf"] = buf
    if own:     # the state that a training program keeps, in the place of its buffers
        import packed_variable_length_gb300 as pvl
        st["state"] = pvl.adamw_state(st["params"], bits=case["bits"], seed=7)
        for key, t in buf.items():
            getattr(st["state"], key).copy_(t)
        st["buf"] = {key: getattr(st["state"], key) for key in buf}
    return st


# --------------------------------------------------------------------- run
def run(st):
    case = st["case"]
    if own:
        return _run_own(st, case)
    if case["op"] == "logprob":
        return _plain_logprob(st, case) if case["dir"] == "fwd" else _plain_logprob_bwd(st, case)
    return {"preference": _plain_preference, "policy": _plain_policy, "adamw": _plain_adamw}[case["op"]](st, case)


def _run_own(st, case):
    import packed_variable_length_gb300 as pvl
    if case["op"] == "logprob":
        if case["dir"] == "fwd":
            out = pvl.pack_logprob_fwd(st["x"], st["t"], st["ids"], temperature=case["T"], entropy=case["entropy"])
            return [t for t in out if t is not None]
        return pvl.pack_logprob_bwd(st["dlogp"], st["x"], st["t"], st["lse"], st["ids"], temperature=case["T"],
                                    ent=st["ent"] if case["entropy"] else None, dent=st["dent"])
    E = case["B"] * case["K"] if "K" in case else 0
    if case["op"] == "preference":
        out = pvl.pack_preference_fwd(st["logp"], st["ref"], st["ids"], st["pairs"], E, kind=case["kind"],
                                      beta=case["beta"], smoothing=case["smoothing"], margin=case["margin"],
                                      mean=case["mean"])
        return out.loss, out.rewards, pvl.pack_preference_bwd(None, out.coef, st["ids"])
    if case["op"] == "policy":
        how = dict(ref_logp=st["ref"], clip_low=case["low"], clip_high=case["high"],
                   kl_weight=case["kl"] if case["ref"] else 0.0, ratio=case["ratio"])
        out = pvl.pack_policy_fwd(st["logp"], st["old"], st["adv"], st["ids"], E, mean=case["mean"], **how)
        return out.loss, out.stats, pvl.pack_policy_bwd(None, st["logp"], st["old"], st["adv"], st["ids"], out.coef, **how)
    norm = pvl.grad_norm(st["grads"]) if case["clip"] else None
    pvl.adamw_step(st["params"], st["grads"], st["state"], LR, betas=BETAS, eps=EPS, weight_decay=DECAY, grad_norm=norm,
                   max_norm=1.0 if case["clip"] else None)
    return _updated(st, norm)


def _updated(st, norm):
    return [t for t in (norm, st["flat"], *(st["buf"][key] for key in sorted(st["buf"]))) if t is not None]


def _live(st, case):
    B, L, V = case["B"], case["L"], case["V"]
    ok = (st["t"] >= 0) & (st["t"] < V)
    return (ok if st["ids"] is None else ok & (st["ids"] >= 0)).view(-1)


def _plain_logprob(st, case):
    V, inv = case["V"], 1.0 / case["T"]
    live = _live(st, case)
    x = st["x"].view(-1, V).float()
    top = x.amax(1, keepdim=True)
    d = (x - top) * inv
    e = d.exp()
    s = e.sum(1, keepdim=True)
    t = st["t"].view(-1, 1).long()
    logs = s.log()
    out = [torch.gather(d, 1, t) - logs, top * inv + logs]
    if case["entropy"]:
        out.append(logs - torch.where(e > 0, e * d, 0.0).sum(1, keepdim=True) / s)
    return [torch.where(live, v[:, 0], 0.0).view(st["t"].shape) for v in out]


def _plain_logprob_bwd(st, case):
    V, inv = case["V"], 1.0 / case["T"]
    live = _live(st, case)[:, None]
    z = st["x"].view(-1, V).float() * inv - st["lse"].view(-1, 1)
    p = z.exp()
    g = st["dlogp"].view(-1, 1)
    out = -g * p
    if case["entropy"]:
        out = out - st["dent"].view(-1, 1) * torch.where(p > 0, p * (z + st["ent"].view(-1, 1)), 0.0)
    t = st["t"].view(-1, 1).long()
    out.scatter_add_(1, t, g)
    return torch.where(live, out * inv, 0.0).to(st["x"].dtype).view(st["x"].shape)


def _slots(st, E):
    """(episode of each token with padding in slot E [N], whether it is valid [N], valid tokens of each episode [E])."""
    ids = st["ids"].view(-1).long()
    valid = ids >= 0
    slot = torch.where(valid, ids, E)
    count = torch.zeros(E + 1, dtype=torch.float64, device="cuda").index_add_(0, slot, valid.double())
    return slot, valid, count[:E]


def _by_episode(v, slot, E):
    """Sums over each episode's tokens: long sums in 64 bits."""
    return torch.zeros(E + 1, dtype=torch.float64, device="cuda").index_add_(0, slot, v.double())[:E]


def _plain_preference(st, case):
    E, beta = case["B"] * case["K"], case["beta"]
    slot, valid, count = _slots(st, E)
    d = st["logp"].view(-1).double() - st["ref"].view(-1).double()
    D = _by_episode(torch.where(valid, d, 0.0), slot, E)
    each = 1.0 / count.clamp(min=1.0) if case["mean"] else torch.ones_like(count)
    D = D * each
    c, r = st["pairs"][:, 0].long(), st["pairs"][:, 1].long()
    h = D[c] - D[r] - case["margin"]
    x = beta * h
    if case["kind"] == "sigmoid":
        s = case["smoothing"]
        soft = torch.log1p(torch.exp(-x.abs()))
        loss = (1.0 - s) * (soft + (-x).clamp(min=0.0)) + s * (soft + x.clamp(min=0.0))
        up = beta * (s - 1.0 / (1.0 + x.exp()))
    elif case["kind"] == "squared":
        loss = (h - 0.5 / beta) ** 2
        up = 2.0 * (h - 0.5 / beta)
    else:
        loss = (1.0 - x).clamp(min=0.0)
        up = torch.where(x < 1.0, -beta, 0.0)
    up = up.double() / case["P"]
    coef = torch.zeros(E, dtype=torch.float64, device="cuda").index_add_(0, c, up).index_add_(0, r, -up) * each
    grad = torch.where(valid, coef[slot.clamp(max=E - 1)], 0.0).float()
    return loss.mean().float().view(1), (beta * D[st["pairs"].long()]).float(), grad.view(st["logp"].shape)


def _plain_policy(st, case):
    E, low, high = case["B"] * case["K"], 1.0 - case["low"], 1.0 + case["high"]
    slot, valid, count = _slots(st, E)
    place = slot.clamp(max=E - 1)
    logp = st["logp"].view(-1)
    d = torch.where(valid, logp.double() - st["old"].view(-1).double(), 0.0)     # 64 bits: values next to the clip border
    live = count > 0
    if case["mean"] == "token":
        weight = torch.ones_like(count) / count.sum().clamp(min=1.0)
    else:
        weight = 1.0 / (count.clamp(min=1.0) * live.sum().clamp(min=1))
    if case["ratio"] == "episode":
        d = _by_episode(d, slot, E) / count.clamp(min=1.0)
        adv = st["adv"].double()
    else:
        adv = (st["adv"].view(-1) if case["adv"] == "token" else st["adv"][place]).double()
    cut = torch.where(adv > 0, d > math.log(high), (adv < 0) & (d < math.log(low)))
    ratio = torch.where(cut, torch.where(adv > 0, high, low), d.exp())
    pg, dpg = -ratio * adv, torch.where(cut, 0.0, -ratio * adv)
    tokens = count.sum().clamp(min=1.0)
    if case["ratio"] == "episode":
        pg, dpg = pg[place], dpg[place]
        share = (cut & live).sum() / live.sum().clamp(min=1)
    else:
        share = (cut & valid).sum() / tokens
    w = torch.where(valid, weight[place], 0.0)
    if case["ref"]:
        f = st["ref"].view(-1).double() - logp.double()     # 64 bits: exp(f) - f - 1 of small f
        kl, dkl = torch.expm1(f) - f, -torch.expm1(f)
    else:
        kl = dkl = torch.zeros((), dtype=torch.float64, device="cuda")
    kl_mean = torch.where(valid, w * kl, 0.0).sum()
    loss = torch.where(valid, w * pg, 0.0).sum() + case["kl"] * kl_mean
    grad = torch.where(valid, w * (dpg + case["kl"] * dkl), 0.0)
    return loss.float().view(1), torch.stack([kl_mean, share.double()]).float(), grad.float().view(st["logp"].shape)


def _mix(z):
    """Wellons' lowbias32 on 32-bit values held in int64."""
    z = z ^ (z >> 16)
    z = (z * 0x7FEB352D) & 0xFFFFFFFF
    z = z ^ (z >> 15)
    z = (z * 0x846CA68B) & 0xFFFFFFFF
    return z ^ (z >> 16)


def _chance(blocks, steps, seed):
    """(u for m, u for v) [blocks, 256] in (0, 1), 16 bits each: vector l of block b hashes b 32 + l with a key of seed
    and step; element j of the vector takes members j and j + 8 of a linear congruential sequence from there."""
    a, c, mul, add = 1, 0, [], []
    for _ in range(16):
        a, c = (a * 1664525) & 0xFFFFFFFF, (c * 1664525 + 1013904223) & 0xFFFFFFFF
        mul.append(a)
        add.append(c)
    mul, add = (torch.tensor(v, device="cuda") for v in (mul, add))
    key = _mix((seed + steps.long() * 0x9E3779B9) & 0xFFFFFFFF)                      # [blocks]
    lane = torch.arange(32, device="cuda")
    h = _mix(((blocks[:, None] * 32 + lane) & 0xFFFFFFFF) ^ key[:, None])            # [blocks, 32]
    r = (h[..., None] * mul + add) & 0xFFFFFFFF                                      # [blocks, 32, 16]
    u = ((r >> 16) * 16 + 8).double() / 2.0 ** 20
    return u[..., :8].reshape(-1, BLOCK), u[..., 8:].reshape(-1, BLOCK)


def _round_e4m3(x, u):
    """x in [-448, 448] to a multiple of its e4m3 step, up with the chance of its remainder."""
    e = torch.frexp(x.abs())[1] - 1
    step = torch.ldexp(torch.ones_like(x), e.clamp(min=-6) - 3)
    q = torch.floor(x.abs() / step + u) * step
    return torch.copysign(q.clamp(max=TOP), x)


def _plain_adamw(st, case):
    places, flat, total = _places(case)
    buf = st["buf"]
    lengths = torch.tensor([-(-n // BLOCK) for n, _, _ in places], device="cuda")
    steps = torch.repeat_interleave(buf["steps"] + 1, lengths)                       # step of each block
    g = torch.zeros(total, device="cuda")
    torch._foreach_copy_([g[a:a + n] for n, _, a in places], [t.view(-1) for t in st["grads"]])
    norm = None
    if case["clip"]:
        norm = g.square().sum(dtype=torch.float64).sqrt().float().view(1)
        g = g * (1.0 / norm).clamp(max=1.0)
    g = g.view(-1, BLOCK)
    if case["bits"] == 8:
        m = buf["m"].float().view(-1, BLOCK) * buf["m_scale"][:, None]
        v = (buf["v"].float().view(-1, BLOCK) * buf["v_scale"][:, None]).square()
    else:
        m, v = buf["m"].view(-1, BLOCK), buf["v"].view(-1, BLOCK)
    b1, b2 = BETAS
    m = m * b1 + g * (1.0 - b1)
    v = v * b2 + g.square() * (1.0 - b2)
    t = steps.double()[:, None]
    first, second = (1.0 - b1 ** t).float(), (1.0 - b2 ** t).sqrt().float()
    root = v.sqrt()
    change = LR / first * (m / (root / second + EPS))
    if "master" in buf:
        p = buf["master"].view(-1, BLOCK)
    else:
        p = torch.zeros(total, device="cuda")
        torch._foreach_copy_([p[a:a + n] for n, _, a in places], [t.view(-1) for t in st["params"]])
        p = p.view(-1, BLOCK)
    p = (p * (1.0 - LR * DECAY) - change).view(-1)
    torch._foreach_copy_([t.view(-1) for t in st["params"]], [p[a:a + n] for n, _, a in places])
    if "master" in buf:
        buf["master"].copy_(p)
    if case["bits"] == 8:
        um, uv = _chance(torch.arange(total // BLOCK, device="cuda"), steps, 7)
        for key, x, u in (("m", m, um), ("v", root, uv)):
            scale = x.abs().amax(1) / TOP
            codes = _round_e4m3(x / torch.where(scale > 0, scale, 1.0)[:, None], u.float())
            if key == "v":
                codes = torch.where(x > 0, codes.clamp(min=2.0 ** -9), codes)
            buf[key].copy_(codes.view(-1))
            buf[key + "_scale"].copy_(scale)
    else:
        buf["m"].copy_(m.view(-1))
        buf["v"].copy_(v.view(-1))
    buf["steps"].add_(1)
    return _updated(st, norm)


# -------------------------------------------------------------------- exact
def exact(case, seed):
    """From the definitions in 64 bits: log-softmax and its derivative, the losses differentiated, the update tensor by
    tensor."""
    st = prepare(case, seed)
    return {"logprob": _exact_logprob, "preference": _exact_preference, "policy": _exact_policy,
            "adamw": _exact_adamw}[case["op"]](st, case)


def _exact_logprob(st, case):
    V, N = case["V"], case["B"] * case["L"]
    rows, t = st["x"].view(N, V), st["t"].view(N).long()
    live = _live(st, case)
    step = max(1, (1 << 26) // V)
    if case["dir"] == "fwd":
        outs = [torch.zeros(N, dtype=torch.float64, device="cuda") for _ in range(3 if case["entropy"] else 2)]
    else:
        grad = torch.zeros(N, V, dtype=torch.float32 if N * V > 1 << 29 else torch.float64, device="cuda")
    for i in range(0, N, step):
        at = i + torch.nonzero(live[i:i + step])[:, 0]
        z = rows[at].double() / case["T"]
        logs = torch.log_softmax(z, 1)
        prob = logs.exp()
        h = -(prob * logs.clamp(min=-1e300)).sum(1)
        if case["dir"] == "fwd":
            outs[0][at] = logs.gather(1, t[at, None])[:, 0]
            outs[1][at] = torch.logsumexp(z, 1)
            if case["entropy"]:
                outs[2][at] = h
            continue
        up = st["dlogp"].view(-1)[at, None].double()
        hot = torch.zeros_like(prob).scatter_(1, t[at, None], 1.0)
        d = up * (hot - prob)
        if case["entropy"]:
            d = d - st["dent"].view(-1)[at, None].double() * prob * (logs.clamp(min=-1e300) + h[:, None])
        grad[at] = (d / case["T"]).to(grad.dtype)
    if case["dir"] == "fwd":
        return [o.view(case["B"], case["L"]) for o in outs]
    return grad.view(case["B"], case["L"], V)


def _member(st, E):
    """[N] tokens of the valid ones and the episode of each."""
    ids = st["ids"].view(-1).long()
    at = torch.nonzero(ids >= 0)[:, 0]
    return at, ids[at]


def _exact_preference(st, case):
    E = case["B"] * case["K"]
    at, who = _member(st, E)
    logp = st["logp"].double().requires_grad_()
    gain = (logp - st["ref"].double()).view(-1)[at]
    total = torch.zeros(E, dtype=torch.float64, device="cuda").index_add(0, who, gain)
    if case["mean"]:
        total = total / torch.bincount(who, minlength=E).clamp(min=1)
    reward = case["beta"] * total
    gap = total[st["pairs"][:, 0].long()] - total[st["pairs"][:, 1].long()] - case["margin"]
    if case["kind"] == "sigmoid":
        s, ls = case["smoothing"], torch.nn.functional.logsigmoid
        loss = -((1 - s) * ls(case["beta"] * gap) + s * ls(-case["beta"] * gap))
    elif case["kind"] == "squared":
        loss = (gap - 1 / (2 * case["beta"])).pow(2)
    else:
        loss = torch.relu(1 - case["beta"] * gap)
    loss = loss.mean()
    grad, = torch.autograd.grad(loss, logp)
    return loss.detach().view(1), reward.detach()[st["pairs"].long()], grad


def _exact_policy(st, case):
    E = case["B"] * case["K"]
    at, who = _member(st, E)
    logp = st["logp"].double().requires_grad_()
    lp = logp.view(-1)[at]
    n = torch.bincount(who, minlength=E).double()
    some = int((n > 0).sum())

    def mean(v):        # of tokens, or of the episodes' means
        if case["mean"] == "token":
            return v.sum() / max(1, v.numel())
        return (torch.zeros(E, dtype=torch.float64, device="cuda").index_add(0, who, v) / n.clamp(min=1)).sum() / max(1, some)

    ratio = lp - st["old"].view(-1)[at].double()
    adv = st["adv"].double() if case["adv"] == "episode" else st["adv"].view(-1)[at].double()
    if case["ratio"] == "episode":
        ratio = torch.zeros(E, dtype=torch.float64, device="cuda").index_add(0, who, ratio) / n.clamp(min=1)
    elif case["adv"] == "episode":
        adv = adv[who]
    ratio = ratio.exp()
    free, held = ratio * adv, ratio.clamp(1 - case["low"], 1 + case["high"]) * adv
    pg, cut = -torch.minimum(free, held), held < free
    if case["ratio"] == "episode":
        share = (cut & (n > 0)).sum() / max(1, some)
        pg = pg[who]
    else:
        share = cut.sum() / max(1, cut.numel())
    kl = torch.zeros((), dtype=torch.float64, device="cuda")
    if case["ref"]:
        f = st["ref"].view(-1)[at].double() - lp
        kl = mean(torch.expm1(f) - f)
    loss = mean(pg) + case["kl"] * kl
    grad, = torch.autograd.grad(loss, logp)
    return loss.detach().view(1), torch.stack([kl.detach(), share.double()]), grad


def _exact_adamw(st, case):
    places, flat, total = _places(case)
    buf, (b1, b2) = st["buf"], BETAS
    size = math.sqrt(sum(float(t.double().square().sum()) for t in st["grads"]))
    held = min(1.0, 1.0 / size) if case["clip"] else 1.0
    t = case["step"] + 1
    new = {key: torch.zeros_like(v, dtype=torch.float64) for key, v in buf.items() if key != "steps"}
    p_new = st["flat"].double()
    for i, (n, f, a) in enumerate(places):
        whole = -(-n // BLOCK) * BLOCK
        g = torch.zeros(whole, dtype=torch.float64, device="cuda")
        g[:n] = st["grads"][i].reshape(-1).double() * held
        m, v = buf["m"][a:a + whole].double(), buf["v"][a:a + whole].double()
        b = slice(a // BLOCK, (a + whole) // BLOCK)
        if case["bits"] == 8:
            m = (m.view(-1, BLOCK) * buf["m_scale"][b, None]).view(-1)
            v = (v.view(-1, BLOCK) * buf["v_scale"][b, None]).view(-1).pow(2)
        m, v = b1 * m + (1 - b1) * g, b2 * v + (1 - b2) * g * g
        p = buf["master"][a:a + n].double() if "master" in buf else st["params"][i].reshape(-1).double()
        p = p - LR * DECAY * p - LR * (m[:n] / (1 - b1 ** t)) / ((v[:n] / (1 - b2 ** t)).sqrt() + EPS)
        p_new[f:f + n] = p
        if "master" in buf:
            new["master"][a:a + n] = p
        if case["bits"] == 32:
            new["m"][a:a + whole], new["v"][a:a + whole] = m, v
            continue
        at = torch.arange(b.start, b.stop, device="cuda")
        chances = _chance(at, torch.full_like(at, t), 7)
        for key, x, u in (("m", m, chances[0]), ("v", v.sqrt(), chances[1])):
            x = x.view(-1, BLOCK)
            scale = x.abs().max(1).values / TOP
            new[key + "_scale"][b] = scale
            y = torch.nan_to_num(x / scale[:, None])
            size_of = y.abs()
            unit = 2.0 ** (torch.floor(torch.log2(size_of.clamp(min=2.0 ** -6))) - 3)
            rest = size_of / unit
            q = (torch.floor(rest) + (rest - torch.floor(rest) + u >= 1.0)) * unit
            q = q.clamp(max=TOP) if key == "m" else torch.where(size_of > 0, q.clamp(2.0 ** -9, TOP), 0.0)
            new[key][a:a + whole] = (q * torch.sign(y)).view(-1)
    new["steps"] = buf["steps"] + 1
    norm = torch.tensor([size], dtype=torch.float64, device="cuda") if case["clip"] else []
    return [norm, p_new, *(new[key] for key in sorted(new))] if case["clip"] else [p_new, *(new[key] for key in sorted(new))]


# --------------------------------------------------------------------- work
def work(case):
    """Bytes that have to move and operations that have to be done in one pass."""
    if case["op"] == "logprob":
        N, V = case["B"] * case["L"], case["V"]
        size = 2 if case["dtype"] == "bf16" else 4
        share = 1.0 - 0.5 * case["pad"]
        ids = 4 * N if case["pad"] else 0
        if case["dir"] == "fwd":
            return {"bytes": share * N * V * size + ids + N * (12 + 4 * case["entropy"]),
                    "flops": share * N * V * (4 + 2 * case["entropy"])}
        return {"bytes": (share + 1.0) * N * V * size + ids + N * (12 + 8 * case["entropy"]),
                "flops": share * N * V * (4 + 4 * case["entropy"])}
    N = case["B"] * case["L"] if "B" in case else 0
    if case["op"] == "preference":
        return {"bytes": 16 * N + 16 * case["P"], "flops": 4 * N + 40 * case["P"]}
    if case["op"] == "policy":
        adv = 4 * N if case["adv"] == "token" else 4 * case["B"] * case["K"]
        return {"bytes": (20 if case["ref"] else 16) * N + adv, "flops": 40 * N}
    n = sum(math.prod(s) for s in _shapes(case))
    each = (8 if case["param"] == "fp32" else 10) + (4 if case["grad"] == "fp32" else 2)
    each += 16 if case["bits"] == 32 else 4 + 16 / BLOCK
    return {"bytes": n * each, "flops": n * (16 if case["bits"] == 32 else 40)}
