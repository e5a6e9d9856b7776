"""torch.autograd wrapper: packed masked attention as a differentiable op.

The tile map is an explicit argument of both passes, so the backward always
sees the mask of its own forward (the class-attribute block-mask hazard of
"lingbot_va_packing" §2.2 cannot occur).
"""

from __future__ import annotations

import torch
from torch.autograd.function import once_differentiable

from . import api


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

