"""Workloads of the operators around packed attention: positions of packed
segments, rotary positions of queries and keys (with the RMS norm before
them), and the gated residual with its norms, in both directions.

Sizes: 12 heads of 128 and the 64k pack are the attention workloads' own,
64,000 x 5120 is the AdaLN workload's, 288 frames of 38 tokens the padded
batch's.
"""

import math

import numpy as np
import torch

own = False

EPS = 1e-6
TOKENS = 38       # tokens per latent frame
ROW = 6           # tokens per image row of a frame (the last row is ragged)


# ------------------------------------------------------------------- cases
def _positions(name, **kw):
    return {"name": name, "op": "positions", **kw}


def _rotary(name, **kw):
    base = {"op": "rotary", "dir": "fwd", "B": 1, "L": 1, "H": 12, "Hk": 12, "D": 128, "R": 128, "axes": 1,
            "layout": "half", "norm": "none", "scaling": "none", "fused": True, "far": 0}
    return {"name": name, **base, **kw}


def _residual(name, **kw):
    base = {"op": "residual", "dir": "fwd", "B": 1, "N": 1, "D": 1536, "mod": "batch", "norm": "layer",
            "post": "none", "affine": False, "stream": "bf16", "alpha": 1.0, "pad": 0}
    return {"name": name, **base, **kw}


def listed():
    return [
        # positions of the four-episode padded batch, as (frame, row, column) for the video tokens
        _positions("positions_padded", B=4, K=1, L=10944, axes=3),
        # positions of the 64k pack of seven episodes, one axis
        _positions("positions_pack64k", B=1, K=7, L=65536, axes=1),
        # one new token for each of eight episodes that run far: serving, latency only
        _rotary("rotary_token", B=8, L=1, fused=False, far=1000000, scaling="parts"),
        # a training step's forward on the 64k pack: q and k normalised over the token, three position axes
        _rotary("rotary_fwd_pack64k", L=65536, axes=3, layout="interleaved", norm="token"),
        # its backward, with the norm weights' gradients
        _rotary("rotary_bwd_pack64k", dir="bwd", L=65536, axes=3, layout="interleaved", norm="token"),
        # shared key heads, part of the head rotated, per-head norm, a ragged length
        _rotary("rotary_fwd_shared", B=3, L=4561, H=16, Hk=4, D=96, R=64, norm="head", scaling="ntk"),
        # the padded batch's backward without a norm
        _rotary("rotary_bwd_padded", dir="bwd", B=4, L=10944),
        # one token of each of eight episodes through the residual and the next norm: serving
        _residual("residual_token", B=8, N=1, D=1536),
        # the AdaLN workload's size as one pack of episodes, each with its own modulation
        _residual("residual_fwd_64k", N=64000, D=5120, mod="episode"),
        _residual("residual_bwd_64k", dir="bwd", N=64000, D=5120, mod="episode"),
        # norms on both sides of the block, an fp32 residual stream, padded rows, a modulation per frame
        _residual("residual_fwd_sandwich", B=4, N=10944, mod="frame", norm="rms", post="rms", affine=True,
                  stream="fp32", alpha=0.75, pad=96),
        _residual("residual_bwd_sandwich", dir="bwd", B=4, N=10944, mod="frame", norm="rms", post="rms", affine=True,
                  stream="fp32", alpha=0.75, pad=96),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["positions", "rotary", "rotary", "residual", "residual"])
    if op == "positions":
        B = _log(rng, 1, 64)
        K = _log(rng, 1, 16)
        L = max(K * TOKENS, _log(rng, 64, 1 << 18) // B)
        return {"op": op, "B": B, "K": K, "L": L, "axes": rng.choice([1, 2, 3])}
    way = rng.choice(["fwd", "bwd"])
    if op == "rotary":
        D = rng.choice([64, 72, 80, 96, 128, 128, 160, 256])
        Hk = rng.choice([1, 2, 3, 4, 6, 12])
        H = Hk * rng.choice([1, 1, 2, 3])
        R = D if rng.random() < 0.6 else 2 * rng.randint(4, D // 2)
        norm = rng.choice(["none", "head", "token"])
        B = _log(rng, 1, 16)
        L = max(1, _log(rng, 1, 60000) // B)
        L = max(1, min(L, 200000000 // (B * (H + Hk) * D)))
        return {"op": op, "dir": way, "B": B, "L": L, "H": H, "Hk": Hk, "D": D, "R": R, "axes": rng.choice([1, 2, 3]),
                "layout": rng.choice(["half", "interleaved"]), "norm": norm,
                "scaling": rng.choice(["none", "linear", "ntk", "parts"]), "fused": rng.random() < 0.5,
                "far": rng.choice([0, 0, 100000, 100000000])}
    D = 8 * _log(rng, 8, 1024)
    B = _log(rng, 1, 16)
    N = max(1, _log(rng, 1, 64000) // B)
    N = max(1, min(N, 160000000 // (B * D)))
    return {"op": op, "dir": way, "B": B, "N": N, "D": D, "mod": rng.choice(["none", "batch", "episode", "frame"]),
            "norm": rng.choice(["layer", "rms"]), "post": rng.choice(["none", "layer", "rms"]),
            "affine": rng.random() < 0.5, "stream": rng.choice(["bf16", "fp32"]),
            "alpha": rng.choice([1.0, 1.0, 0.5]), "pad": rng.choice([0, 0, 17])}


# ------------------------------------------------------------------- inputs
def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _randn(g, *shape, dtype=torch.float32, mul=1.0, add=0.0):
    out = torch.empty(shape, dtype=dtype, device="cuda")
    step = max(1, (1 << 27) // max(1, out[0].numel()))
    for i in range(0, shape[0], step):      # in pieces: the fp32 draw of a large tensor need not be whole
        part = out[i:i + step]
        part.copy_(torch.randn(part.shape, generator=g, device="cuda").mul_(mul).add_(add))
    return out


def _segment_frames(case, seed):
    """[B, K] frame counts, whole frames laid end to end within L."""
    rng = np.random.default_rng(seed)
    cap = case["L"] // TOKENS
    cuts = np.sort(rng.integers(0, cap + 1, size=(case["B"], case["K"])), axis=1)
    cuts[:, -1] = np.maximum(cuts[:, -1], cap - rng.integers(0, 8, size=case["B"]).clip(max=cap // 2))
    cuts = np.sort(cuts, axis=1)
    return np.diff(cuts, axis=1, prepend=0).astype(np.int32)


def _sections(R, axes):
    """Pairs of each position axis: the first takes what is left over."""
    part = (R // 2) // axes
    return (R // 2 - part * (axes - 1),) + (part,) * (axes - 1)


def _angular(case):
    """(frequencies in radians per position [R/2], axis of each pair, gain): one ladder per axis."""
    kind, factor, length, base = case["scaling"], 4.0, 4096, 10000.0
    freqs, axis, gain = [], [], 1.0
    for a, n in enumerate(_sections(case["R"], case["axes"])):
        b = base * factor ** (n / (n - 1.0)) if kind == "ntk" and n > 1 else base
        f = b ** (-np.arange(n, dtype=np.float64) / max(n, 1))
        if kind == "linear":
            f = f / factor
        if kind == "parts":
            turns = length * f / (2.0 * math.pi)
            keep = np.clip((turns - 1.0) / (32.0 - 1.0), 0.0, 1.0)
            f = f * keep + f / factor * (1.0 - keep)
            gain = 0.1 * math.log(factor) + 1.0
        freqs.append(f)
        axis.append(np.full(n, a))
    return np.concatenate(freqs), np.concatenate(axis), gain


def _heads(g, case, H):
    return _randn(g, case["B"], case["L"], H, case["D"], dtype=torch.bfloat16)


def _valid_frames(case):
    """Whole frames of each batch row that are real: row b has pad * b // B fewer than the row holds."""
    F = -(-case["N"] // TOKENS)
    return [max(0, F - case["pad"] * (b + 1) // case["B"]) if case["pad"] else F for b in range(case["B"])]


def _mod_rows(case):
    if case["mod"] in ("none", "batch"):
        return case["B"]
    F = -(-case["N"] // TOKENS)
    return case["B"] * (F if case["mod"] == "frame" else min(7, F))


def _mod_id(case, seed):
    """int32 [B, N]: the modulation row of each token, -1 on padding; None where it is the batch row."""
    if case["mod"] in ("none", "batch") and not case["pad"]:
        return None
    B, N = case["B"], case["N"]
    F = -(-N // TOKENS)
    frame = np.arange(N) // TOKENS
    rng = np.random.default_rng(seed)
    ids = np.empty((B, N), dtype=np.int32)
    for b, valid in enumerate(_valid_frames(case)):
        if case["mod"] == "frame":
            row = b * F + frame
        elif case["mod"] == "episode":
            K = min(7, F)
            starts = np.sort(rng.integers(0, F, size=K))
            starts[0] = 0
            row = b * K + np.searchsorted(starts, frame, side="right") - 1
        else:
            row = np.full(N, b)
        ids[b] = np.where(frame < valid, row, -1)
    return torch.from_numpy(ids).cuda()


def prepare(case, seed):
    if case["op"] == "positions":
        return {"case": case, "frames": _segment_frames(case, seed)}
    g = _gen(seed)
    if case["op"] == "rotary":
        B, L, H, Hk, D, R = (case[k] for k in ("B", "L", "H", "Hk", "D", "R"))
        st = {"case": case}
        if case["fused"]:       # q, k (and v) are slices of one projection's output
            qkv = _randn(g, B, L, H + 2 * Hk, D, dtype=torch.bfloat16)
            st["q"], st["k"] = qkv[:, :, :H], qkv[:, :, H:H + Hk]
        else:
            st["q"], st["k"] = _heads(g, case, H), _heads(g, case, Hk)
        if case["dir"] == "bwd":
            st["dq"], st["dk"] = _heads(g, case, H), _heads(g, case, Hk)
        wide = case["norm"] == "token"
        st["wq"] = st["wk"] = None
        if case["norm"] != "none":
            st["wq"] = _randn(g, H * D if wide else D, mul=0.1, add=1.0)
            st["wk"] = _randn(g, Hk * D if wide else D, mul=0.1, add=1.0)
        # positions restart in each packed episode, or go on from far behind
        step = torch.randint(0, 362, (B, L, case["axes"]), generator=g, device="cuda", dtype=torch.int32)
        start = torch.randint(0, case["far"] + 1, (B, 1, case["axes"]), generator=g, device="cuda", dtype=torch.int32)
        st["pos"] = start + step
        f, axis, st["gain"] = _angular(case)
        st["freq"], st["axis"] = torch.from_numpy(f).cuda(), torch.from_numpy(axis).cuda()
        if own:     # the plan that a model keeps for all its layers and steps
            import packed_variable_length_gb300 as pvl
            st["plan"] = pvl.rotary_plan(R, layout=case["layout"], sections=_sections(R, case["axes"]),
                                         scaling=case["scaling"], factor=4.0, length=4096, device="cuda")
        return st
    B, N, D = case["B"], case["N"], case["D"]
    S = _mod_rows(case)
    xt = torch.float32 if case["stream"] == "fp32" else torch.bfloat16
    st = {"case": case, "ids": _mod_id(case, seed)}
    # a residual stream has a common offset and a larger spread than what the block adds
    st["x"] = _randn(g, B, N, D, dtype=xt, mul=2.0, add=0.5)
    st["h"] = _randn(g, B, N, D, dtype=torch.bfloat16)
    mod = case["mod"] != "none"
    st["gate"] = _randn(g, S, D, mul=0.5) if mod else None
    st["shift"] = _randn(g, S, D, mul=0.5) if mod else None
    st["scale"] = _randn(g, S, D, mul=0.3) if mod else None
    st["w"] = _randn(g, D, mul=0.1, add=1.0) if case["affine"] else None
    st["b"] = _randn(g, D, mul=0.1) if case["affine"] and case["norm"] == "layer" else None
    st["w2"] = _randn(g, D, mul=0.1, add=1.0) if case["post"] != "none" else None
    if case["dir"] == "bwd":
        st["dx_out"] = _randn(g, B, N, D, dtype=xt)
        st["dy"] = _randn(g, B, N, D, dtype=torch.bfloat16)
    return st


# --------------------------------------------------------------------- run
def run(st):
    case = st["case"]
    if own:
        return _run_own(st, case)
    if case["op"] == "positions":
        return _plain_positions(st, case)
    if case["op"] == "rotary":
        return _plain_rotary(st, case) if case["dir"] == "fwd" else _plain_rotary_bwd(st, case)
    return _plain_residual(st, case) if case["dir"] == "fwd" else _plain_residual_bwd(st, case)


def _run_own(st, case):
    import packed_variable_length_gb300 as pvl
    if case["op"] == "positions":
        return pvl.pack_build_positions(st["frames"], TOKENS, case["L"], axes=case["axes"],
                                        row_width=ROW if case["axes"] == 3 else None)
    if case["op"] == "rotary":
        norm = None if case["norm"] == "none" else case["norm"]
        if case["dir"] == "fwd":
            return pvl.pack_rotary_fwd(st["q"], st["k"], st["pos"], st["plan"], norm=norm, q_weight=st["wq"],
                                       k_weight=st["wk"], eps=EPS)
        out = pvl.pack_rotary_bwd(st["dq"], st["dk"], st["pos"], st["plan"], norm=norm, q=st["q"], k=st["k"],
                                  q_weight=st["wq"], k_weight=st["wk"], eps=EPS)
        return [t for t in out if t is not None]
    how = dict(mod_id=st["ids"], weight=st["w"], bias=st["b"], post_weight=st["w2"], norm=case["norm"],
               post_norm=None if case["post"] == "none" else case["post"], alpha=case["alpha"], eps=EPS)
    if case["dir"] == "fwd":
        return pvl.adaln_residual_fwd(st["x"], st["h"], st["gate"], st["shift"], st["scale"], **how)
    out = pvl.adaln_residual_bwd(st["dx_out"], st["dy"], st["x"], st["h"], st["gate"], st["shift"], st["scale"], **how)
    return [t for t in out if t is not None]


def _plain_positions(st, case):
    """Each token's offset from the start of its segment, split into axes."""
    L = case["L"]
    ends = torch.from_numpy(st["frames"]).cuda().long().cumsum(1) * TOKENS         # [B, K]
    p = torch.arange(L, device="cuda").expand(case["B"], L).contiguous()
    k = torch.searchsorted(ends, p, right=True)                                    # segments that end at or before p
    inside = k < case["K"]
    starts = torch.cat([torch.zeros_like(ends[:, :1]), ends], dim=1)
    i = torch.where(inside, p - torch.gather(starts, 1, k), torch.zeros_like(p))
    frame, slot = i // TOKENS, i % TOKENS
    if case["axes"] == 1:
        out = i[:, :, None]
    elif case["axes"] == 2:
        out = torch.stack([frame, slot], dim=2)
    else:
        out = torch.stack([frame, slot // ROW, slot % ROW], dim=2)
    return out.to(torch.int32)


def _cos_sin(st):
    angle = st["pos"][:, :, st["axis"]].double() * st["freq"]           # [B, L, R/2]: 64 bits for far positions
    return ((angle.cos() * st["gain"]).float()[:, :, None], (angle.sin() * st["gain"]).float()[:, :, None])


def _rotate(x, cos, sin, case):
    """x fp32 [B, L, H, D]: the first R features of each head turned, the rest as they are."""
    R = case["R"]
    if case["layout"] == "half":
        a, b = x[..., :R // 2], x[..., R // 2:R]
        turned = torch.cat([a * cos - b * sin, a * sin + b * cos], dim=-1)
    else:
        a, b = x[..., 0:R:2], x[..., 1:R:2]
        turned = torch.stack([a * cos - b * sin, a * sin + b * cos], dim=-1).flatten(-2)
    return torch.cat([turned, x[..., R:]], dim=-1)


def _rms(x, case):
    """(x / rms, 1 / rms) over the head or over all heads of the token."""
    over = (2, 3) if case["norm"] == "token" else (3,)
    r = torch.rsqrt(x.square().mean(over, keepdim=True) + EPS)
    return x * r, r


def _weight(w, x, case):
    return w.view(x.shape[2:]) if case["norm"] == "token" else w


def _plain_rotary(st, case):
    cos, sin = _cos_sin(st)

    def one(x, w):
        x = x.float()
        if w is not None:
            x = _rms(x, case)[0] * _weight(w, x, case)
        return _rotate(x, cos, sin, case).to(torch.bfloat16)

    return one(st["q"], st["wq"]), one(st["k"], st["wk"])


def _plain_rotary_bwd(st, case):
    cos, sin = _cos_sin(st)

    def one(x, dout, w):
        g = _rotate(dout.float(), cos, -sin, case)
        if w is None:
            return g.to(torch.bfloat16), None
        xh, r = _rms(x.float(), case)
        dw = (g * xh).sum((0, 1)).flatten() if case["norm"] == "token" else (g * xh).sum((0, 1, 2))
        g = g * _weight(w, g, case)
        over = (2, 3) if case["norm"] == "token" else (3,)
        dx = r * (g - xh * (g * xh).mean(over, keepdim=True))
        return dx.to(torch.bfloat16), dw

    dq, dwq = one(st["q"], st["dq"], st["wq"])
    dk, dwk = one(st["k"], st["dk"], st["wk"])
    return [t for t in (dq, dk, dwq, dwk) if t is not None]


def _norm(x, kind):
    """(x normalised, 1 / deviation) over the features."""
    if kind == "layer":
        x = x - x.mean(2, keepdim=True)
    r = torch.rsqrt(x.square().mean(2, keepdim=True) + EPS)
    return x * r, r


def _norm_bwd(g, xh, r, kind):
    out = g - xh * (g * xh).mean(2, keepdim=True)
    return (out - g.mean(2, keepdim=True) if kind == "layer" else out) * r


def _tables(st, case):
    """(row of each token [B, N] with padding on row 0, whether it is real [B, N, 1], pick of a table's rows)."""
    B, N = case["B"], case["N"]
    ids = st["ids"]
    if ids is None:
        ids = torch.arange(B, device="cuda")[:, None].expand(B, N)
    real = (ids >= 0)[:, :, None]
    row = ids.clamp(min=0).long()
    return row, real, (lambda t: t[row])


def _plain_residual(st, case):
    row, real, pick = _tables(st, case)
    x, u = st["x"].float(), st["h"].float()
    if case["post"] != "none":
        u = _norm(u, case["post"])[0] * st["w2"]
    if st["gate"] is not None:
        u = u * pick(st["gate"])
    t = torch.where(real, case["alpha"] * x + u, x)
    y = _norm(t, case["norm"])[0]
    if st["w"] is not None:
        y = y * st["w"]
    if st["b"] is not None:
        y = y + st["b"]
    if st["scale"] is not None:
        y = y * (1.0 + pick(st["scale"])) + pick(st["shift"])
    return t.to(st["x"].dtype), torch.where(real, y, torch.zeros_like(y)).to(torch.bfloat16)


def _plain_residual_bwd(st, case):
    row, real, pick = _tables(st, case)
    zero = torch.zeros((), device="cuda")
    dxo, dy = st["dx_out"].float(), torch.where(real, st["dy"].float(), zero)
    h = torch.where(real, st["h"].float(), zero)
    xh, r = _norm(st["x"].float(), case["norm"])
    hot = torch.nn.functional.one_hot(row.flatten(), _mod_rows(case)).float().t()        # [S, B N]

    def by_row(v):                                  # sums over each modulation row's tokens
        return hot @ v.reshape(-1, case["D"])

    s1 = 1.0 + pick(st["scale"]) if st["scale"] is not None else torch.ones((), device="cuda")
    n = xh if st["w"] is None else xh * st["w"]
    n = n if st["b"] is None else n + st["b"]
    dshift = by_row(dy) if st["shift"] is not None else None
    dscale = by_row(dy * n) if st["scale"] is not None else None
    dn = dy * s1
    dw = (dn * xh).sum((0, 1)) if st["w"] is not None else None
    db = dn.sum((0, 1)) if st["b"] is not None else None
    t = dxo + _norm_bwd(dn if st["w"] is None else dn * st["w"], xh, r, case["norm"])
    t = torch.where(real, t, dxo)
    dx = torch.where(real, case["alpha"] * t, t)
    du = torch.where(real, t, zero)
    hh, rh = (h, None) if case["post"] == "none" else _norm(h, case["post"])
    u = hh if st["w2"] is None else hh * st["w2"]
    dgate = by_row(du * u) if st["gate"] is not None else None
    if st["gate"] is not None:
        du = du * pick(st["gate"])
    dw2 = (du * hh).sum((0, 1)) if st["w2"] is not None else None
    if st["w2"] is not None:
        du = du * st["w2"]
    dh = du if rh is None else _norm_bwd(du, hh, rh, case["post"])
    out = (dx.to(st["x"].dtype), dh.to(torch.bfloat16), dgate, dshift, dscale, dw, db, dw2)
    return [v for v in out if v is not None]


# -------------------------------------------------------------------- exact
def exact(case, seed):
    """From the definitions in 64 bits: rotation as a product of complex
    numbers, gradients by differentiating the forward."""
    st = prepare(case, seed)
    if case["op"] == "positions":
        return None
    if case["op"] == "rotary":
        return _exact_rotary(st, case)
    return _exact_residual(st, case)


def _exact_rotary(st, case):
    R, D = case["R"], case["D"]
    angle = st["pos"].double()[:, :, st["axis"]] * st["freq"][None, None]
    turn = torch.polar(torch.full_like(angle, st["gain"]), angle)[:, :, None]

    def forward(x, w):
        if w is not None:
            flat = x.flatten(2) if case["norm"] == "token" else x
            flat = flat / (flat.pow(2).sum(-1, keepdim=True) / flat.shape[-1] + EPS).sqrt() * w
            x = flat.reshape(x.shape)
        pairs = x[..., :R].reshape(*x.shape[:3], 2, R // 2).transpose(3, 4) if case["layout"] == "half" \
            else x[..., :R].reshape(*x.shape[:3], R // 2, 2)
        z = torch.complex(pairs[..., 0].contiguous(), pairs[..., 1].contiguous()) * turn
        z = torch.view_as_real(z)
        z = z.transpose(3, 4) if case["layout"] == "half" else z
        return torch.cat([z.reshape(*x.shape[:3], R), x[..., R:]], -1)

    def one(x, w, dout):
        x = x.double()
        w = None if w is None else w.double()
        if dout is None:
            return forward(x, w), None
        leaves = [x.requires_grad_()] + ([] if w is None else [w.requires_grad_()])
        grads = torch.autograd.grad(forward(x, w), leaves, dout.double())
        return grads[0], grads[1] if w is not None else None

    q, wq = one(st["q"], st["wq"], st.get("dq"))
    k, wk = one(st["k"], st["wk"], st.get("dk"))
    return [t for t in (q, k, wq, wk) if t is not None]


def _exact_residual(st, case):
    B, N, D = case["B"], case["N"], case["D"]
    ids = st["ids"]
    if ids is None:
        ids = torch.arange(B, device="cuda", dtype=torch.int32)[:, None].repeat(1, N)
    ids = ids.reshape(-1)
    live = torch.nonzero(ids >= 0)[:, 0]
    row = ids[live].long()

    def wide(key):
        return None if st.get(key) is None else st[key].double()

    def rows(key):
        return st[key].reshape(-1, D)[live].double()

    def normalise(v, kind):
        centre = v.mean(1, keepdim=True) if kind == "layer" else 0.0
        spread = ((v - centre) ** 2).mean(1, keepdim=True)
        return (v - centre) / (spread + EPS).sqrt()

    def branch(h, gate, w2):
        u = h if case["post"] == "none" else normalise(h, case["post"]) * w2
        return u if gate is None else u * gate.index_select(0, row)

    def outer(t, w, b, scale, shift):
        n = normalise(t, case["norm"])
        n = n if w is None else n * w
        n = n if b is None else n + b
        return n if scale is None else n + n * scale.index_select(0, row) + shift.index_select(0, row)

    if case["dir"] == "fwd":
        t = case["alpha"] * rows("x") + branch(rows("h"), wide("gate"), wide("w2"))
        x_out = st["x"].reshape(-1, D).double().index_copy(0, live, t)
        y = torch.zeros_like(x_out).index_copy(0, live, outer(t, wide("w"), wide("b"), wide("scale"), wide("shift")))
        return x_out.view(B, N, D), y.view(B, N, D)

    def grads(f, args, upstream):
        on = [a.requires_grad_() for a in args if a is not None]
        got = iter(torch.autograd.grad(f(*args), on, upstream))
        return [None if a is None else next(got) for a in args]

    dt, dw, db, dscale, dshift = grads(outer, [rows("x"), wide("w"), wide("b"), wide("scale"), wide("shift")], rows("dy"))
    dt = dt + rows("dx_out")
    dh, dgate, dw2 = grads(branch, [rows("h"), wide("gate"), wide("w2")], dt)
    dx = st["dx_out"].reshape(-1, D).double().index_copy(0, live, case["alpha"] * dt)
    dh = torch.zeros_like(dx).index_copy(0, live, dh)
    out = (dx.view(B, N, D), dh.view(B, N, D), dgate, dshift, dscale, dw, db, dw2)
    return [v for v in out if v is not None]


# --------------------------------------------------------------------- work
def work(case):
    """Bytes that have to move and operations that have to be done in one pass."""
    if case["op"] == "positions":
        n = case["B"] * case["L"]
        return {"bytes": 4 * n * case["axes"] + 4 * case["B"] * case["K"], "flops": 6 * n}
    if case["op"] == "rotary":
        tokens = case["B"] * case["L"]
        each = tokens * (case["H"] + case["Hk"]) * case["D"]
        norm = case["norm"] != "none"
        tensors = 2 if case["dir"] == "fwd" or not norm else 3
        weights = 0
        if norm:
            weights = (case["H"] + case["Hk"]) * case["D"] if case["norm"] == "token" else 2 * case["D"]
            weights *= 1 if case["dir"] == "fwd" else 2
        per = (4 if case["dir"] == "fwd" else 12) if norm else 0
        return {"bytes": 2 * tensors * each + 4 * tokens * case["axes"] + 4 * weights,
                "flops": each * (4 + per) + 10 * tokens * case["R"]}
    B, N, D = case["B"], case["N"], case["D"]
    frames = torch.tensor(_valid_frames(case))
    live = int((frames * TOKENS).clamp(max=N).sum())
    dead = B * N - live
    xb = 4 if case["stream"] == "fp32" else 2
    tables = 3 * _mod_rows(case) * D if case["mod"] != "none" else 0
    vectors = D * (int(case["affine"]) + int(case["affine"] and case["norm"] == "layer") + int(case["post"] != "none"))
    needs_h = case["mod"] != "none" or case["post"] != "none"
    if case["dir"] == "fwd":
        each = live * (2 * xb + 4) + dead * (2 * xb + 2)
        par, ops = tables + vectors, 14
    else:
        each = live * (3 * xb + 4 + (2 if needs_h else 0)) + dead * (2 * xb + 2)
        par, ops = 2 * (tables + vectors), 30
    ids = 4 * B * N if case["pad"] or case["mod"] in ("episode", "frame") else 0
    return {"bytes": each * D + 4 * par + ids, "flops": ops * live * D + (8 * live * D if case["post"] != "none" else 0)}
