"""torch.autograd wrapper: packed masked attention as a differentiable op.

The tile map is an explicit argument of both passes, so the backward always
sees the mask of its own forward (the class-attribute block-mask hazard of
"lingbot_va_packing" §2.2 cannot occur).
"""

from __future__ import annotations

import torch
from torch.autograd.function import once_differentiable

from . import api, objectives


class _PackedAttention(torch.autograd.Function):
    @staticmethod
    def forward(ctx, q, k, v, seq_id, k_seq_id, tile_map, scale):
        o, lse = api.masked_attn_fwd(q, k, v, seq_id, tile_map, scale, k_seq_id=k_seq_id)
        ctx.save_for_backward(q, k, v, o, lse, seq_id, k_seq_id)
        ctx.tile_map = tile_map
        ctx.scale = scale
        return o

    @staticmethod
    def backward(ctx, do):
        q, k, v, o, lse, seq_id, k_seq_id = ctx.saved_tensors
        dq, dk, dv = api.masked_attn_bwd(q, k, v, o, do.contiguous(), lse, seq_id, ctx.tile_map, ctx.scale,
                                         k_seq_id=k_seq_id)
        return dq, dk, dv, None, None, None, None


def packed_attention(q, k, v, seq_id, tile_map=None, scale=None, k_seq_id=None):
    """O = masked softmax attention of bf16 [B, L, H, D] q/k/v under int32 [B, L]
    seq_id; with k_seq_id (int32 [B, Lk]) cross attention of q [B, L, H, D]
    against k, v [B, Lk, H, D] ("lingbot_va_packing" §2.1)."""
    if tile_map is None:
        tile_map = api.tile_map_build(seq_id, k_seq_id=k_seq_id)
    return _PackedAttention.apply(q, k, v, seq_id, k_seq_id, tile_map, scale)


class _AdaLNModulate(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, shift, scale, eps):
        y = api.adaln_fwd(x, shift, scale, eps)
        ctx.save_for_backward(x, scale)
        ctx.eps = eps
        return y

    @staticmethod
    def backward(ctx, dy):
        x, scale = ctx.saved_tensors
        dx, dshift, dscale = api.adaln_bwd(x, scale, dy.contiguous(), ctx.eps)
        return dx, dshift, dscale, None


def adaln_modulate(x, shift, scale, eps: float = 1e-6):
    """layer_norm(x) * (1 + scale) + shift over bf16 x [B, N, D] with fp32
    shift / scale [B, D], differentiable ("AdaptiveLoad" §2.B); the backward
    recomputes the row statistics from x."""
    return _AdaLNModulate.apply(x, shift, scale, eps)


class _PackedRotary(torch.autograd.Function):
    @staticmethod
    def forward(ctx, q, k, positions, plan, norm, q_weight, k_weight, eps):
        q_out, k_out = api.pack_rotary_fwd(q, k, positions, plan, norm, q_weight, k_weight, eps)
        normed = norm is not None
        ctx.save_for_backward(q if normed else None, k if normed else None, positions, q_weight, k_weight)
        ctx.how = (plan, norm, eps)
        return q_out if k is None else (q_out, k_out)

    @staticmethod
    @once_differentiable
    def backward(ctx, dq_out, dk_out=None):
        q, k, positions, q_weight, k_weight = ctx.saved_tensors
        plan, norm, eps = ctx.how
        dq_out, dk_out = (t if t is None or t.stride(3) == 1 else t.contiguous() for t in (dq_out, dk_out))
        dq, dk, dqw, dkw = api.pack_rotary_bwd(dq_out, dk_out, positions, plan, norm, q, k, q_weight, k_weight, eps)
        return dq, dk, None, None, None, dqw, dkw, None


def packed_rotary(q, k, positions, plan, norm=None, q_weight=None, k_weight=None, eps: float = 1e-6):
    """Rotary positions of bf16 q [B, L, H, D] and k [B, L, Hk, D] (k may be
    None: the result is then the rotated q alone), with the RMS norm before
    them, differentiable in q, k and the norm weights (see
    api.pack_rotary_fwd); the outputs are what packed_attention takes."""
    return _PackedRotary.apply(q, k, positions, plan, norm, q_weight, k_weight, eps)


def _dense(t):
    """t contiguous and on a 16-byte boundary, where a gradient that comes as a part of another need not be."""
    t = t.contiguous()
    return t if t.data_ptr() % 16 == 0 else t.clone()


class _GatedResidual(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, h, gate, shift, scale, weight, bias, post_weight, mod_id, how):
        x_out, y = api.adaln_residual_fwd(x, h, gate, shift, scale, mod_id=mod_id, weight=weight, bias=bias,
                                          post_weight=post_weight, **how)
        # without a gate or a post norm no gradient depends on h
        kept = h if h is not None and (gate is not None or how["post_norm"] is not None) else None
        ctx.save_for_backward(x_out, kept, gate, shift, scale, weight, bias, post_weight, mod_id)
        ctx.how = how
        ctx.branch = h is not None
        ctx.set_materialize_grads(False)
        return y if h is None else (x_out, y)

    @staticmethod
    @once_differentiable
    def backward(ctx, *grads):
        x_out, h, gate, shift, scale, weight, bias, post_weight, mod_id = ctx.saved_tensors
        dx_out, dy = grads if ctx.branch else (None, grads[0])
        if dy is None:
            dy = torch.zeros(x_out.shape, dtype=torch.bfloat16, device=x_out.device)
        if dx_out is not None:
            dx_out = _dense(dx_out)
        g = api.adaln_residual_bwd(dx_out, _dense(dy), x_out, h, gate, shift, scale, mod_id=mod_id, weight=weight,
                                   bias=bias, post_weight=post_weight, branch=ctx.branch, **ctx.how)
        return (*g, None, None)


def gated_residual(x, h=None, gate=None, shift=None, scale=None, *, mod_id=None, weight=None, bias=None,
                   post_weight=None, norm: str = "layer", post_norm: str | None = None, alpha: float = 1.0,
                   eps: float = 1e-6):
    """(x_out, y) of api.adaln_residual_fwd, differentiable in every floating
    input: the gated residual after a block and the modulated norm before the
    next, with one modulation row per packed episode (mod_id).  Without h,
    x_out is x itself."""
    how = dict(norm=norm, post_norm=post_norm, alpha=alpha, eps=eps)
    out = _GatedResidual.apply(x, h, gate, shift, scale, weight, bias, post_weight, mod_id, how)
    return (x, out) if h is None else out


class _MaskedMSE(torch.autograd.Function):
    @staticmethod
    def forward(ctx, pred, target, seq_id):
        loss = api.masked_mse_loss(pred, target, seq_id)
        ctx.save_for_backward(pred, target, seq_id)
        return loss.view(())

    @staticmethod
    def backward(ctx, dloss):
        pred, target, seq_id = ctx.saved_tensors
        grad = api.masked_mse_loss_bwd(pred, target, seq_id, dloss.reshape(1).contiguous())
        return grad, None, None


def frame_valid_mse(pred, target, seq_id):
    """Squared-error loss of bf16 pred [B, L, C] against target, averaged
    over the valid tokens (seq_id >= 0: the valid frames), differentiable in
    pred ("lingbot_va_packing" §2.1, compute_loss).  The backward reads pred
    and target again and scales by the incoming gradient on the device."""
    return _MaskedMSE.apply(pred, target, seq_id)



class _TokenLogprob(torch.autograd.Function):
    @staticmethod
    def forward(ctx, logits, targets, seq_id, temperature, entropy):
        logp, lse, ent = objectives.pack_logprob_fwd(logits, targets, seq_id, temperature=temperature, entropy=entropy)
        ctx.save_for_backward(logits, targets, seq_id, lse, ent)
        ctx.temperature = temperature
        ctx.set_materialize_grads(False)
        return (logp, ent) if entropy else logp

    @staticmethod
    @once_differentiable
    def backward(ctx, dlogp, dent=None):
        logits, targets, seq_id, lse, ent = ctx.saved_tensors
        if dlogp is None and dent is None:
            return None, None, None, None, None
        dlogp, dent = (None if t is None else t.contiguous() for t in (dlogp, dent))
        return objectives.pack_logprob_bwd(dlogp, logits, targets, lse, seq_id, temperature=ctx.temperature, ent=ent,
                                           dent=dent), None, None, None, None


def token_logprob(logits, targets, seq_id=None, *, temperature: float = 1.0, entropy: bool = False):
    """fp32 [B, L] log-probabilities of targets under logits [B, L, V] (see
    objectives.pack_logprob_fwd), with entropy=True (log-probabilities, entropy
    of each row), differentiable in the logits."""
    return _TokenLogprob.apply(logits, targets, seq_id, temperature, entropy)


def _constants(op: str, **tensors) -> None:
    """What an op takes as given may not ask for a gradient, which would be lost."""
    if torch.is_grad_enabled():
        for name, t in tensors.items():
            if isinstance(t, torch.Tensor) and t.requires_grad:
                raise ValueError(f"{op} gives no gradient to {name}, which requires one: pass {name}.detach()")


class _PreferenceLoss(torch.autograd.Function):
    @staticmethod
    def forward(ctx, logp, ref_logp, seq_id, pairs, episodes, how):
        out = objectives.pack_preference_fwd(logp, ref_logp, seq_id, pairs, episodes, **how)
        ctx.save_for_backward(out.coef, seq_id)
        ctx.mark_non_differentiable(out.rewards)
        return out.loss.view(()), out.rewards

    @staticmethod
    @once_differentiable
    def backward(ctx, dloss, _):
        coef, seq_id = ctx.saved_tensors
        return (objectives.pack_preference_bwd(dloss.reshape(1).contiguous(), coef, seq_id),) + (None,) * 5


def preference_loss(logp, ref_logp, seq_id, pairs, episodes: int, *, beta: float = 0.1, kind: str = "sigmoid",
                    smoothing: float = 0.0, margin: float = 0.0, mean: bool = False):
    """(loss, rewards) of objectives.pack_preference_fwd: the preference loss
    over pairs of packed episodes, differentiable in logp, and the rewards of
    each pair's episodes.  ref_logp is taken as given: one that requires a
    gradient is refused."""
    _constants("preference_loss", ref_logp=ref_logp)
    how = dict(beta=beta, kind=kind, smoothing=smoothing, margin=margin, mean=mean)
    return _PreferenceLoss.apply(logp, ref_logp, seq_id, pairs, episodes, how)


class _PolicyLoss(torch.autograd.Function):
    @staticmethod
    def forward(ctx, logp, old_logp, advantages, seq_id, ref_logp, episodes, mean, how):
        out = objectives.pack_policy_fwd(logp, old_logp, advantages, seq_id, episodes, ref_logp=ref_logp, mean=mean,
                                         **how)
        ctx.save_for_backward(logp, old_logp, advantages, seq_id, ref_logp, out.coef)
        ctx.how = how
        ctx.mark_non_differentiable(out.stats)
        return out.loss.view(()), out.stats

    @staticmethod
    @once_differentiable
    def backward(ctx, dloss, _):
        logp, old_logp, advantages, seq_id, ref_logp, coef = ctx.saved_tensors
        return (objectives.pack_policy_bwd(dloss.reshape(1).contiguous(), logp, old_logp, advantages, seq_id, coef,
                                           ref_logp=ref_logp, **ctx.how),) + (None,) * 7


def policy_loss(logp, old_logp, advantages, seq_id, episodes: int, *, ref_logp=None, clip_low: float = 0.2,
                clip_high: float = 0.2, kl_weight: float = 0.0, ratio: str = "token", mean: str = "token"):
    """(loss, stats) of objectives.pack_policy_fwd: the clipped policy loss with
    its divergence term, differentiable in logp, and (divergence, share of
    clipped ratios).  What it is measured against (old_logp, advantages,
    ref_logp) is taken as given: tensors that require a gradient are refused."""
    _constants("policy_loss", old_logp=old_logp, advantages=advantages, ref_logp=ref_logp)
    how = dict(clip_low=clip_low, clip_high=clip_high, kl_weight=kl_weight, ratio=ratio)
    return _PolicyLoss.apply(logp, old_logp, advantages, seq_id, ref_logp, episodes, mean, how)
