"""Python binding of the losses of a packed policy: log-probabilities of tokens
from logits, the preference loss over pairs of episodes and the clipped policy
loss, with their gradients.

As in api.py, every function checks its arguments, allocates what the caller
does not pass on the current stream, and calls the C entry point of the same
name; all arithmetic runs in the library's kernels.
"""

from __future__ import annotations

from typing import NamedTuple

import torch

from . import _lib
from .api import _addr, _check, _launch, _need, _need_cuda, _ptr


# ------------------------------------------------------- log-probabilities
def _row_strides(t, name: str):
    """(batch stride, token stride) of [B, L, V] rows that are dense; the stride of a single entry means nothing."""
    B, L, V = t.shape
    sb, sl, sv = t.stride()
    if sv != 1 and V > 1:
        raise ValueError(f"{name} must be contiguous in its last dimension")
    return sb if B > 1 else 0, sl if L > 1 else 0


def _logprob(logits, targets, seq_id, temperature):
    """Checked description of a log-probability call."""
    if not isinstance(logits, torch.Tensor) or logits.dim() != 3:
        raise ValueError("logits must be [B, L, V]")
    if logits.dtype not in (torch.bfloat16, torch.float32):
        raise ValueError(f"logits must be {torch.bfloat16} or {torch.float32}, got {logits.dtype}")
    B, L, V = logits.shape
    dev = logits.device
    if not isinstance(targets, torch.Tensor) or targets.dtype not in (torch.int32, torch.int64):
        raise ValueError(f"targets must be {torch.int32} or {torch.int64}")
    _need(targets, "targets", targets.dtype, (B, L), dev)
    if seq_id is not None:
        _need(seq_id, "seq_id", torch.int32, (B, L), dev)
    sb, sl = _row_strides(logits, "logits")
    return _lib.PACK_LOGPROB(B, L, V, 1 if logits.dtype is torch.float32 else 0,
                             1 if targets.dtype is torch.int64 else 0, float(temperature), logits.data_ptr(),
                             targets.data_ptr(), _addr(seq_id), sb, sl)


def pack_logprob_fwd(logits, targets, seq_id=None, *, temperature: float = 1.0, entropy: bool = False, logp=None,
                     lse=None, ent=None, stream=None):
    """(logp, lse, entropy): fp32 [B, L] log-probability of each int32 or int64
    target [B, L] under softmax(logits / temperature) of bf16 or fp32 logits
    [B, L, V], the log of each row's normaliser and, with entropy=True, the
    entropy of each row (else None).

    Rows may have any strides (logits[:, :-1], or a padded vocabulary's
    logits[..., :V]).  Tokens whose seq_id (int32 [B, L], optional) is negative
    or whose target lies outside [0, V) give zeros and are not read."""
    how = _logprob(logits, targets, seq_id, temperature)
    dev, shape = logits.device, targets.shape
    with _launch(dev, stream) as handle:
        out = []
        for name, t, wanted in (("logp", logp, True), ("lse", lse, True), ("ent", ent, entropy)):
            if not wanted:
                t = None
            elif t is None:
                t = torch.empty(shape, dtype=torch.float32, device=dev)
            else:
                _need(t, name, torch.float32, shape, dev)
            out.append(t)
        _check(_lib.load().pack_logprob_fwd(how, out[0].data_ptr(), out[1].data_ptr(), _ptr(out[2]), handle))
    return tuple(out)


def pack_logprob_bwd(dlogp, logits, targets, lse, seq_id=None, *, temperature: float = 1.0, ent=None, dent=None,
                     dlogits=None, stream=None):
    """Gradient of pack_logprob_fwd to the logits, of their type: from dlogp
    (fp32 [B, L], or None for zero) and, with dent, from the gradient of the
    entropy (which needs ent, the forward's).  dlogits, where given, may have
    strides of its own; it may be the logits, which are then overwritten."""
    how = _logprob(logits, targets, seq_id, temperature)
    dev, shape = logits.device, targets.shape
    if dlogp is None and dent is None:
        raise ValueError("dlogp or dent must be given")
    if dent is not None and ent is None:
        raise ValueError("the gradient of the entropy needs ent")
    for name, t in (("dlogp", dlogp), ("lse", lse), ("ent", ent), ("dent", dent)):
        if t is not None or name == "lse":
            _need(t, name, torch.float32, shape, dev)
    if dlogits is not None:
        if not isinstance(dlogits, torch.Tensor) or dlogits.dtype is not logits.dtype or (
                dlogits.shape != logits.shape or dlogits.device != dev):
            raise ValueError(f"dlogits must be {logits.dtype} {tuple(logits.shape)} on {dev}")
    with _launch(dev, stream) as handle:
        if dlogits is None:
            dlogits = torch.empty(logits.shape, dtype=logits.dtype, device=dev)
        sb, sl = _row_strides(dlogits, "dlogits")
        _check(_lib.load().pack_logprob_bwd(how, lse.data_ptr(), _ptr(ent), _ptr(dlogp), _ptr(dent),
                                            dlogits.data_ptr(), sb, sl, handle))
    return dlogits


# ------------------------------------------------------------- preference
_PREFERENCES = {"sigmoid": 0, "squared": 1, "hinge": 2}


class PreferenceLoss(NamedTuple):
    """Results of pack_preference_fwd."""
    loss: torch.Tensor      # fp32 [1]
    rewards: torch.Tensor   # fp32 [P, 2]: beta times the log ratio of the chosen and of the rejected episode
    coef: torch.Tensor      # fp32 [episodes]: d loss / d logp of each episode's tokens


def _tokens(logp, seq_id):
    """Checks the tokens of a pack, of any shape; returns (device, shape)."""
    if not isinstance(seq_id, torch.Tensor):
        raise ValueError("seq_id must be a tensor")
    _need_cuda(seq_id, "seq_id", torch.int32)
    if logp is not None:
        _need(logp, "logp", torch.float32, seq_id.shape, seq_id.device)
    return seq_id.device, seq_id.shape


def _workspace(ws, nbytes: int, dev):
    if ws is None:
        return torch.empty(max(nbytes, 1), dtype=torch.uint8, device=dev)
    _need(ws, "ws", torch.uint8, ws.shape, dev)
    return ws


def pack_preference_ws_bytes(episodes: int) -> int:
    return int(_lib.load().pack_preference_ws_bytes(int(episodes)))


def pack_preference_fwd(logp, ref_logp, seq_id, pairs, episodes: int, *, beta: float = 0.1, kind: str = "sigmoid",
                        smoothing: float = 0.0, margin: float = 0.0, mean: bool = False, ws=None,
                        stream=None) -> PreferenceLoss:
    """Preference loss over int32 pairs [P, 2] of (chosen, rejected) episodes of
    a pack.  logp and ref_logp (or None) are fp32 like seq_id (int32; the ids of
    pack_build_seq_ids, below `episodes`, negative for tokens that take no
    part): the log-probability of each token, or any other log-likelihood that
    adds up over an episode, such as minus a squared error.

    With D the sum over an episode of logp - ref_logp (mean=True: their mean)
    and h = D[chosen] - D[rejected] - margin, the loss is the mean over pairs of
    "sigmoid": -(1 - smoothing) log sigmoid(beta h) - smoothing log
    sigmoid(-beta h); "squared": (h - 1 / (2 beta))^2; "hinge": max(0, 1 - beta
    h).  A pair with a negative id is left out."""
    dev, shape = _tokens(logp, seq_id)
    if logp is None:
        raise ValueError("logp must be given")
    if ref_logp is not None:
        _need(ref_logp, "ref_logp", torch.float32, shape, dev)
    if kind not in _PREFERENCES:
        raise ValueError(f"kind must be one of {sorted(_PREFERENCES)}, got {kind!r}")
    if not isinstance(pairs, torch.Tensor) or pairs.dim() != 2 or pairs.shape[1] != 2:
        raise ValueError("pairs must be [P, 2]")
    _need(pairs, "pairs", torch.int32, pairs.shape, dev)
    E, P = int(episodes), int(pairs.shape[0])
    how = _lib.PACK_PREFERENCE(seq_id.numel(), E, P, _PREFERENCES[kind], int(bool(mean)), float(beta),
                               float(smoothing), float(margin), logp.data_ptr(), _addr(ref_logp), seq_id.data_ptr(),
                               pairs.data_ptr())
    lib = _lib.load()
    with _launch(dev, stream) as handle:
        ws = _workspace(ws, int(lib.pack_preference_ws_bytes(E)), dev)
        out = torch.empty(1 + 2 * P + max(E, 1), dtype=torch.float32, device=dev)
        loss, rewards, coef = out[:1], out[1:1 + 2 * P].view(P, 2), out[1 + 2 * P:]
        _check(lib.pack_preference_fwd(how, loss.data_ptr(), rewards.data_ptr(), coef.data_ptr(), ws.data_ptr(),
                                       ws.numel(), handle))
    return PreferenceLoss(loss, rewards, coef)


def pack_preference_bwd(dloss, coef, seq_id, *, dlogp=None, stream=None):
    """d loss / d logp (fp32 like seq_id) from coef of pack_preference_fwd, times
    the device scalar dloss (fp32, one element; None for 1)."""
    dev, shape = _tokens(None, seq_id)
    if not isinstance(coef, torch.Tensor) or coef.dim() != 1:
        raise ValueError("coef must be [episodes]")
    _need(coef, "coef", torch.float32, coef.shape, dev)
    _scalar(dloss, dev)
    with _launch(dev, stream) as handle:
        dlogp = _like_tokens(dlogp, shape, dev)
        _check(_lib.load().pack_preference_bwd(_ptr(dloss), coef.data_ptr(), seq_id.data_ptr(), seq_id.numel(),
                                               coef.shape[0], dlogp.data_ptr(), handle))
    return dlogp


def _scalar(dloss, dev):
    if dloss is None:
        return
    if not isinstance(dloss, torch.Tensor) or dloss.numel() != 1:
        raise ValueError("dloss must hold one element")
    _need(dloss, "dloss", torch.float32, dloss.shape, dev)


def _like_tokens(t, shape, dev):
    if t is None:
        return torch.empty(shape, dtype=torch.float32, device=dev)
    _need(t, "dlogp", torch.float32, shape, dev)
    return t


# ----------------------------------------------------------------- policy
class PolicyLoss(NamedTuple):
    """Results of pack_policy_fwd."""
    loss: torch.Tensor      # fp32 [1]
    stats: torch.Tensor     # fp32 [2]: divergence from the reference, share of clipped ratios
    coef: torch.Tensor      # fp32 [episodes, 2], for pack_policy_bwd


_OVER = {"token": 0, "episode": 1}


def _policy(logp, old_logp, advantages, seq_id, episodes, ref_logp, clip_low, clip_high, kl_weight, ratio, mean):
    dev, shape = _tokens(logp, seq_id)
    if logp is None:
        raise ValueError("logp must be given")
    for name, t in (("old_logp", old_logp), ("ref_logp", ref_logp)):
        if t is not None:
            _need(t, name, torch.float32, shape, dev)
    for name, v in (("ratio", ratio), ("mean", mean)):
        if v not in _OVER:
            raise ValueError(f"{name} must be 'token' or 'episode', got {v!r}")
    if not isinstance(advantages, torch.Tensor):
        raise ValueError("advantages must be a tensor")
    tokens = ratio == "token" and advantages.shape == shape
    _need(advantages, "advantages", torch.float32, shape if tokens else (int(episodes),), dev)
    return _lib.PACK_POLICY(seq_id.numel(), int(episodes), _OVER[ratio], _OVER[mean], int(tokens), float(clip_low),
                            float(clip_high), float(kl_weight), logp.data_ptr(), _addr(old_logp), _addr(ref_logp),
                            advantages.data_ptr(), seq_id.data_ptr()), dev, shape


def pack_policy_ws_bytes(episodes: int) -> int:
    return int(_lib.load().pack_policy_ws_bytes(int(episodes)))


def pack_policy_fwd(logp, old_logp, advantages, seq_id, episodes: int, *, ref_logp=None, clip_low: float = 0.2,
                    clip_high: float = 0.2, kl_weight: float = 0.0, ratio: str = "token", mean: str = "token",
                    ws=None, stream=None) -> PolicyLoss:
    """Clipped policy loss with a divergence term over the tokens of a pack that
    have an id (seq_id >= 0; ids below `episodes`).  logp, old_logp (None: logp
    itself, a ratio of 1) and ref_logp are fp32 like seq_id; advantages fp32
    like seq_id, or one an episode, [episodes].

    With r = exp(logp - old_logp) (ratio="episode": exp of the mean over the
    token's episode, which needs advantages of episodes) a token's loss is
    -min(r A, clip(r, 1 - clip_low, 1 + clip_high) A) + kl_weight (exp(f) - f -
    1), f = ref_logp - logp; the loss is their mean (mean="episode": the mean of
    the episodes' means)."""
    how, dev, _ = _policy(logp, old_logp, advantages, seq_id, episodes, ref_logp, clip_low, clip_high, kl_weight,
                          ratio, mean)
    E = int(episodes)
    lib = _lib.load()
    with _launch(dev, stream) as handle:
        ws = _workspace(ws, int(lib.pack_policy_ws_bytes(E)), dev)
        out = torch.empty(4 + 2 * max(E, 1), dtype=torch.float32, device=dev)
        loss, stats, coef = out[:1], out[1:3], out[4:].view(-1, 2)
        _check(lib.pack_policy_fwd(how, loss.data_ptr(), stats.data_ptr(), coef.data_ptr(), ws.data_ptr(), ws.numel(),
                                   handle))
    return PolicyLoss(loss, stats, coef)


def pack_policy_bwd(dloss, logp, old_logp, advantages, seq_id, coef, *, ref_logp=None, clip_low: float = 0.2,
                    clip_high: float = 0.2, kl_weight: float = 0.0, ratio: str = "token", dlogp=None, stream=None):
    """d loss / d logp (fp32 like seq_id) of pack_policy_fwd from the same inputs
    and its coef, times the device scalar dloss (fp32, one element; None for 1)."""
    if not isinstance(coef, torch.Tensor) or coef.dim() != 2 or coef.shape[1] != 2:
        raise ValueError("coef must be [episodes, 2]")
    how, dev, shape = _policy(logp, old_logp, advantages, seq_id, coef.shape[0], ref_logp, clip_low, clip_high,
                              kl_weight, ratio, "token")
    _need(coef, "coef", torch.float32, coef.shape, dev)
    _scalar(dloss, dev)
    with _launch(dev, stream) as handle:
        dlogp = _like_tokens(dlogp, shape, dev)
        _check(_lib.load().pack_policy_bwd(how, _ptr(dloss), coef.data_ptr(), dlogp.data_ptr(), handle))
    return dlogp
