"""Python binding of the losses of a packed policy: log-probabilities of tokens
from logits, the preference loss over pairs of episodes and the clipped policy
loss, with their gradients.

As in api.py, every function checks its arguments, allocates what the caller
does not pass on the current stream, and calls the C entry point of the same
name; all arithmetic runs in the library's kernels.
"""

from __future__ import annotations

from functools import lru_cache
from typing import NamedTuple

import torch

from . import _lib
from .api import _addr, _check, _here, _launch, _need, _need_cuda, _ptr

_F32, _BF16, _I32, _I64 = torch.float32, torch.bfloat16, torch.int32, torch.int64


def _tensor(t, name: str, dtype, shape, dev) -> None:
    """api._need, without a call where the tensor's type says the rest (these calls take microseconds)."""
    if t.dtype is not dtype or t.shape != shape or t.device != dev or not t.is_contiguous():
        _need(t, name, dtype, shape, dev)


# ------------------------------------------------------- log-probabilities
def _row_strides(t, name: str):
    """(batch stride, token stride) of [B, L, V] rows that are dense; the stride of a single entry means nothing."""
    B, L, V = t.shape
    sb, sl, sv = t.stride()
    if sv != 1 and V > 1:
        raise ValueError(f"{name} must be contiguous in its last dimension")
    return sb if B > 1 else 0, sl if L > 1 else 0


def _kind(t, name: str, kinds) -> int:
    """Which of two types a tensor has: 0 or 1."""
    if isinstance(t, torch.Tensor):
        if t.dtype is kinds[0]:
            return 0
        if t.dtype is kinds[1]:
            return 1
        raise ValueError(f"{name} must be {kinds[0]} or {kinds[1]}, got {t.dtype}")
    raise ValueError(f"{name} must be a tensor")


def _logprob(logits, targets, seq_id, temperature):
    """Checked description of a log-probability call."""
    wide = _kind(logits, "logits", (_BF16, _F32))
    if logits.dim() != 3:
        raise ValueError("logits must be [B, L, V]")
    long = _kind(targets, "targets", (_I32, _I64))
    B, L, V = logits.shape
    dev, shape = logits.device, (B, L)
    _tensor(targets, "targets", targets.dtype, shape, dev)
    if seq_id is not None:
        _need(seq_id, "seq_id", _I32, shape, dev)
    sb, sl = _row_strides(logits, "logits")
    return _lib.PACK_LOGPROB(B, L, V, wide, long, temperature, logits.data_ptr(), targets.data_ptr(), _addr(seq_id),
                             sb, sl), dev, shape


def _rows(t, name: str, shape, dev):
    if t is None:
        return torch.empty(shape, dtype=_F32, device=dev)
    _need(t, name, _F32, shape, dev)
    return t


def pack_logprob_fwd(logits, targets, seq_id=None, *, temperature: float = 1.0, entropy: bool = False, logp=None,
                     lse=None, ent=None, stream=None):
    """(logp, lse, entropy): fp32 [B, L] log-probability of each int32 or int64
    target [B, L] under softmax(logits / temperature) of bf16 or fp32 logits
    [B, L, V], the log of each row's normaliser and, with entropy=True, the
    entropy of each row (else None).

    Rows may have any strides (logits[:, :-1], or a padded vocabulary's
    logits[..., :V]); targets and seq_id have to be contiguous.  Tokens whose
    seq_id (int32 [B, L], optional) is negative or whose target lies outside
    [0, V) give zeros and are not read."""
    how, dev, shape = _logprob(logits, targets, seq_id, temperature)
    handle = _here(dev, stream)
    if handle is None:
        with _launch(dev, stream) as handle:
            return _run_logprob(how, dev, shape, logp, lse, ent, entropy, handle)
    return _run_logprob(how, dev, shape, logp, lse, ent, entropy, handle)


def _wrote(*outputs) -> None:
    """Counts the outputs that a caller gave (None for the others) as changed in place, as autograd has it for its own:
    a graph that needs what they held refuses to go on."""
    torch.autograd.graph.increment_version([t for t in outputs if t is not None])


def _run_logprob(how, dev, shape, logp, lse, ent, entropy, handle):
    given = (logp, lse, ent if entropy else None) if logp is not None or lse is not None or ent is not None else None
    logp, lse = _rows(logp, "logp", shape, dev), _rows(lse, "lse", shape, dev)
    ent = _rows(ent, "ent", shape, dev) if entropy else None
    _check(_lib.load().pack_logprob_fwd(how, logp.data_ptr(), lse.data_ptr(), _ptr(ent), handle))
    if given is not None:
        _wrote(*given)
    return logp, lse, ent


def pack_logprob_bwd(dlogp, logits, targets, lse, seq_id=None, *, temperature: float = 1.0, ent=None, dent=None,
                     dlogits=None, stream=None):
    """Gradient of pack_logprob_fwd to the logits, of their type: from dlogp
    (fp32 [B, L], or None for zero) and, with dent, from the gradient of the
    entropy (which needs ent, the forward's).  dlogits, where given, may have
    strides of its own; it may be the logits, which are then overwritten (a
    change in place to autograd), but not otherwise reach into them."""
    how, dev, shape = _logprob(logits, targets, seq_id, temperature)
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
    handle = _here(dev, stream)
    if handle is None:
        with _launch(dev, stream) as handle:
            return _run_logprob_bwd(how, logits, lse, ent, dlogp, dent, dlogits, handle)
    return _run_logprob_bwd(how, logits, lse, ent, dlogp, dent, dlogits, handle)


def _run_logprob_bwd(how, logits, lse, ent, dlogp, dent, dlogits, handle):
    given = dlogits
    if dlogits is None:
        dlogits = torch.empty(logits.shape, dtype=logits.dtype, device=logits.device)
    sb, sl = _row_strides(dlogits, "dlogits")
    _check(_lib.load().pack_logprob_bwd(how, lse.data_ptr(), _ptr(ent), _ptr(dlogp), _ptr(dent), dlogits.data_ptr(),
                                        sb, sl, handle))
    if given is not None:
        _wrote(given)
    return dlogits


# ------------------------------------------------------------- preference
_PREFERENCES = {"sigmoid": 0, "squared": 1, "hinge": 2}


class PreferenceLoss(NamedTuple):
    """Results of pack_preference_fwd."""
    loss: torch.Tensor      # fp32 [1]
    rewards: torch.Tensor   # fp32 [P, 2]: beta times the log ratio of the chosen and of the rejected episode
    coef: torch.Tensor      # fp32 [episodes]: d loss / d logp of each episode's tokens


def _tokens(seq_id):
    """Checks the ids of a pack, of any shape; returns (device, shape)."""
    if not isinstance(seq_id, torch.Tensor) or seq_id.dtype is not _I32 or not seq_id.is_contiguous() or (
            not seq_id.is_cuda):
        _need_cuda(seq_id, "seq_id", _I32)
    return seq_id.device, seq_id.shape


def _of_tokens(shape, dev, **tensors) -> None:
    """Says which of the tensors (None where they are left out) is not fp32, of the shape, contiguous, on the device."""
    for name, t in tensors.items():
        if t is None and name != "logp":
            continue
        if not isinstance(t, torch.Tensor):
            raise ValueError(f"{name} must be a tensor")
        if t.dtype is not _F32 or t.shape != shape or t.device != dev or not t.is_contiguous():
            _need(t, name, _F32, shape, dev)


@lru_cache(maxsize=256)
def _preference_ws_bytes(episodes: int) -> int:
    return int(_lib.load().pack_preference_ws_bytes(episodes))


@lru_cache(maxsize=256)
def _policy_ws_bytes(episodes: int) -> int:
    return int(_lib.load().pack_policy_ws_bytes(episodes))


def _workspace(ws, nbytes: int, dev):
    if ws is None:
        return torch.empty(max(nbytes, 1), dtype=torch.uint8, device=dev)
    _need(ws, "ws", torch.uint8, ws.shape, dev)
    return ws


def pack_preference_ws_bytes(episodes: int) -> int:
    return _preference_ws_bytes(int(episodes))


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
    dev, shape = _tokens(seq_id)
    _of_tokens(shape, dev, logp=logp, ref_logp=ref_logp)
    if kind not in _PREFERENCES:
        raise ValueError(f"kind must be one of {sorted(_PREFERENCES)}, got {kind!r}")
    if not isinstance(pairs, torch.Tensor) or pairs.dim() != 2 or pairs.shape[1] != 2:
        raise ValueError("pairs must be [P, 2]")
    _tensor(pairs, "pairs", _I32, pairs.shape, dev)
    E, P = int(episodes), pairs.shape[0]
    how = _lib.PACK_PREFERENCE(seq_id.numel(), E, P, _PREFERENCES[kind], 1 if mean else 0, beta, smoothing, margin,
                               logp.data_ptr(), _addr(ref_logp), seq_id.data_ptr(), pairs.data_ptr())
    handle = _here(dev, stream)
    if handle is None:
        with _launch(dev, stream) as handle:
            return _run_preference(how, dev, E, P, ws, handle)
    return _run_preference(how, dev, E, P, ws, handle)


def _run_preference(how, dev, E, P, ws, handle):
    ws = _workspace(ws, _preference_ws_bytes(E), dev)
    loss = torch.empty(1, dtype=_F32, device=dev)
    rewards = torch.empty((P, 2), dtype=_F32, device=dev)
    coef = torch.empty(max(E, 1), dtype=_F32, device=dev)
    _check(_lib.load().pack_preference_fwd(how, loss.data_ptr(), rewards.data_ptr(), coef.data_ptr(), ws.data_ptr(),
                                           ws.numel(), handle))
    return PreferenceLoss(loss, rewards, coef)


def pack_preference_bwd(dloss, coef, seq_id, *, dlogp=None, stream=None):
    """d loss / d logp (fp32 like seq_id) from coef of pack_preference_fwd, times
    the device scalar dloss (fp32, one element; None for 1)."""
    dev, shape = _tokens(seq_id)
    if not isinstance(coef, torch.Tensor) or coef.dim() != 1:
        raise ValueError("coef must be [episodes]")
    _tensor(coef, "coef", _F32, coef.shape, dev)
    if dloss is not None:
        _scalar(dloss, dev)
    handle = _here(dev, stream)
    if handle is None:
        with _launch(dev, stream) as handle:
            return _run_preference_bwd(dloss, coef, seq_id, dlogp, shape, dev, handle)
    return _run_preference_bwd(dloss, coef, seq_id, dlogp, shape, dev, handle)


def _run_preference_bwd(dloss, coef, seq_id, dlogp, shape, dev, handle):
    given = dlogp
    dlogp = _rows(dlogp, "dlogp", shape, dev)
    _check(_lib.load().pack_preference_bwd(_ptr(dloss), coef.data_ptr(), seq_id.data_ptr(), seq_id.numel(),
                                           coef.shape[0], dlogp.data_ptr(), handle))
    if given is not None:
        _wrote(given)
    return dlogp


def _scalar(dloss, dev):
    if not isinstance(dloss, torch.Tensor) or dloss.numel() != 1:
        raise ValueError("dloss must hold one element")
    _need(dloss, "dloss", torch.float32, dloss.shape, dev)


# ----------------------------------------------------------------- policy
class PolicyLoss(NamedTuple):
    """Results of pack_policy_fwd."""
    loss: torch.Tensor      # fp32 [1]
    stats: torch.Tensor     # fp32 [2]: divergence from the reference, share of clipped ratios
    coef: torch.Tensor      # fp32 [episodes, 2], for pack_policy_bwd


_OVER = {"token": 0, "episode": 1}


def _policy(logp, old_logp, advantages, seq_id, episodes, ref_logp, clip_low, clip_high, kl_weight, ratio, mean):
    dev, shape = _tokens(seq_id)
    _of_tokens(shape, dev, logp=logp, old_logp=old_logp, ref_logp=ref_logp)
    if ratio not in _OVER or mean not in _OVER:
        raise ValueError(f"ratio and mean must be 'token' or 'episode', got {ratio!r} and {mean!r}")
    if not isinstance(advantages, torch.Tensor):
        raise ValueError("advantages must be a tensor")
    tokens = ratio == "token" and advantages.shape == shape
    _tensor(advantages, "advantages", _F32, shape if tokens else (episodes,), dev)
    return _lib.PACK_POLICY(seq_id.numel(), episodes, _OVER[ratio], _OVER[mean], 1 if tokens else 0, clip_low, clip_high,
                            kl_weight, logp.data_ptr(), _addr(old_logp), _addr(ref_logp), advantages.data_ptr(),
                            seq_id.data_ptr()), dev, shape


def pack_policy_ws_bytes(episodes: int) -> int:
    return _policy_ws_bytes(int(episodes))


def pack_policy_fwd(logp, old_logp, advantages, seq_id, episodes: int, *, ref_logp=None, clip_low: float = 0.2,
                    clip_high: float = 0.2, kl_weight: float = 0.0, ratio: str = "token", mean: str = "token",
                    ws=None, stream=None) -> PolicyLoss:
    """Clipped policy loss with a divergence term over the tokens of a pack that
    have an id (seq_id >= 0; ids below `episodes`).  logp, old_logp (None: logp
    itself, a ratio of 1) and ref_logp are fp32 like seq_id; advantages fp32
    like seq_id, or one an episode, [episodes] (where both shapes are the same:
    of tokens with ratio="token", of episodes with ratio="episode").

    With r = exp(logp - old_logp) (ratio="episode": exp of the mean over the
    token's episode, which needs advantages of episodes) a token's loss is
    -min(r A, clip(r, 1 - clip_low, 1 + clip_high) A) + kl_weight (exp(f) - f -
    1), f = ref_logp - logp; the loss is their mean (mean="episode": the mean of
    the episodes' means)."""
    E = int(episodes)
    how, dev, _ = _policy(logp, old_logp, advantages, seq_id, E, ref_logp, clip_low, clip_high, kl_weight, ratio, mean)
    handle = _here(dev, stream)
    if handle is None:
        with _launch(dev, stream) as handle:
            return _run_policy(how, dev, E, ws, handle)
    return _run_policy(how, dev, E, ws, handle)


def _run_policy(how, dev, E, ws, handle):
    ws = _workspace(ws, _policy_ws_bytes(E), dev)
    loss = torch.empty(1, dtype=_F32, device=dev)
    stats = torch.empty(2, dtype=_F32, device=dev)
    coef = torch.empty((max(E, 1), 2), dtype=_F32, device=dev)
    _check(_lib.load().pack_policy_fwd(how, loss.data_ptr(), stats.data_ptr(), coef.data_ptr(), ws.data_ptr(),
                                       ws.numel(), handle))
    return PolicyLoss(loss, stats, coef)


def pack_policy_bwd(dloss, logp, old_logp, advantages, seq_id, coef, *, ref_logp=None, clip_low: float = 0.2,
                    clip_high: float = 0.2, kl_weight: float = 0.0, ratio: str = "token", dlogp=None, stream=None):
    """d loss / d logp (fp32 like seq_id) of pack_policy_fwd from the same inputs
    and its coef, times the device scalar dloss (fp32, one element; None for 1)."""
    if not isinstance(coef, torch.Tensor) or coef.dim() != 2 or coef.shape[1] != 2:
        raise ValueError("coef must be [episodes, 2]")
    how, dev, shape = _policy(logp, old_logp, advantages, seq_id, coef.shape[0], ref_logp, clip_low, clip_high,
                              kl_weight, ratio, "token")
    _tensor(coef, "coef", _F32, coef.shape, dev)
    if dloss is not None:
        _scalar(dloss, dev)
    handle = _here(dev, stream)
    if handle is None:
        with _launch(dev, stream) as handle:
            return _run_policy_bwd(how, dloss, coef, dlogp, shape, dev, handle)
    return _run_policy_bwd(how, dloss, coef, dlogp, shape, dev, handle)


def _run_policy_bwd(how, dloss, coef, dlogp, shape, dev, handle):
    given = dlogp
    dlogp = _rows(dlogp, "dlogp", shape, dev)
    _check(_lib.load().pack_policy_bwd(how, _ptr(dloss), coef.data_ptr(), dlogp.data_ptr(), handle))
    if given is not None:
        _wrote(given)
    return dlogp
