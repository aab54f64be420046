"""torch.autograd wrappers: the provider's outputs with gradients attached.

Page "feat(rl-kernel): add CUDA linear logp provider integration", Summary and
Changes: the provider returns log probabilities and optional entropy, and the
caller rejects detached gradients, so both outputs must carry gradients back to
whatever produced them - the hidden states, projection weight and bias on the fused
route, or the reused logits on the logits-reuse route.

Each forward runs one library call and keeps its merged LSE and entropy for the
backward, which is again one library call (three tcgen05 GEMMs plus reductions on the
fused route, one streaming kernel on the logits route). Nothing here computes: the
wrappers only route tensors between the two calls.

    logp, entropy = linear_logp(X, [W], None, part, y, tau)
    (logp * advantages).sum().backward()       # X.grad, W.grad

The operator's neighbours in a training step have wrappers of the same kind: embedding,
policy_loss and preference_loss.

    X = block(embedding(ids, [W], part))
    logp, entropy = linear_logp(X, [W], None, part, y, tau)
    loss, metrics, counts = policy_loss(logp, old_logp, advantages, entropy=entropy, entropy_coef=1e-3)
    loss.backward()
"""
from __future__ import annotations

from typing import Optional, Sequence

import torch
from torch.autograd.function import once_differentiable

from . import (lp_backward_ex, lp_backward_from_logits, lp_embedding, lp_embedding_backward, lp_forward,
               lp_forward_from_logits, lp_policy_loss, lp_preference_loss)


def _zeros_like_rows(ref: torch.Tensor) -> torch.Tensor:
    return torch.zeros(ref.shape[0], dtype=torch.float32, device=ref.device)


def _f32(g: Optional[torch.Tensor]) -> Optional[torch.Tensor]:
    return None if g is None else g.to(torch.float32).contiguous()


class _LinearLogp(torch.autograd.Function):
    @staticmethod
    def forward(ctx, X, part, y, tau, n, has_bias, *wb):
        W = list(wb[:n])
        bias = list(wb[n:]) if has_bias else None
        out = lp_forward(X, W, bias, part, y, tau, entropy=True)
        ctx.part, ctx.tau, ctx.n, ctx.has_bias = part, tau, n, has_bias
        ctx.save_for_backward(X, y, out["lse"], out["entropy"], *wb)
        ctx.mark_non_differentiable(out["lse"])
        ctx.set_materialize_grads(False)
        return out["logp"], out["entropy"], out["lse"]

    @staticmethod
    def backward(ctx, g_logp, g_entropy, _g_lse):
        X, y, lse, entropy, *wb = ctx.saved_tensors
        n = ctx.n
        W = wb[:n]
        bias = wb[n:] if ctx.has_bias else None
        if g_logp is None and g_entropy is None:
            return (None,) * (6 + len(wb))
        g = _f32(g_logp) if g_logp is not None else _zeros_like_rows(X)
        want_db = bias is not None and any(b is not None and b.requires_grad for b in bias)
        # X and W are bf16, so their gradients are bf16: the library rounds its fp32 results
        # once, as autograd's own cast would, and writes half the bytes
        r = lp_backward_ex(X, W, bias, ctx.part, y, ctx.tau, lse, g, bias_grad=want_db,
                           entropy=entropy if g_entropy is not None else None, grad_entropy=_f32(g_entropy),
                           dx_dtype=torch.bfloat16, dw_dtype=torch.bfloat16)
        dX = r["dX"] if ctx.needs_input_grad[0] else None
        dW = [d if ctx.needs_input_grad[6 + k] else None for k, d in enumerate(r["dW"])]
        db = [None] * n
        if want_db:
            db = [d if ctx.needs_input_grad[6 + n + k] else None for k, d in enumerate(r["db"])]
        return (dX, None, None, None, None, None, *dW, *(db if ctx.has_bias else []))


def linear_logp(X: torch.Tensor, W: Sequence[torch.Tensor], bias: Optional[Sequence[torch.Tensor]], part,
                y: torch.Tensor, tau: float):
    """Fused linear-logp with autograd: returns (logp, entropy), both differentiable with
    respect to X, every W[k] and every bias[k]. The merged LSE is kept for the backward."""
    n = len(part.ranges)
    if len(W) != n:
        raise ValueError("W must have one entry per shard")
    wb = list(W) + (list(bias) if bias is not None else [])
    logp, entropy, _ = _LinearLogp.apply(X, part, y, float(tau), n, bias is not None, *wb)
    return logp, entropy


class _LinearLogpFromLogits(torch.autograd.Function):
    @staticmethod
    def forward(ctx, part, y, tau, *logits):
        out = lp_forward_from_logits(list(logits), part, y, tau, entropy=True)
        ctx.part, ctx.tau = part, tau
        ctx.save_for_backward(y, out["lse"], out["entropy"], *logits)
        ctx.mark_non_differentiable(out["lse"])
        ctx.set_materialize_grads(False)
        return out["logp"], out["entropy"], out["lse"]

    @staticmethod
    def backward(ctx, g_logp, g_entropy, _g_lse):
        y, lse, entropy, *logits = ctx.saved_tensors
        if g_logp is None and g_entropy is None:
            return (None,) * (3 + len(logits))
        g = _f32(g_logp) if g_logp is not None else _zeros_like_rows(y)
        dL = lp_backward_from_logits(logits, ctx.part, y, ctx.tau, lse, g,
                                     entropy=entropy if g_entropy is not None else None,
                                     grad_entropy=_f32(g_entropy), out_dtype=torch.bfloat16)
        return (None, None, None, *[d if ctx.needs_input_grad[3 + k] else None for k, d in enumerate(dL)])


def linear_logp_from_logits(logits: Sequence[torch.Tensor], part, y: torch.Tensor, tau: float):
    """Logits-reuse linear-logp with autograd: returns (logp, entropy), differentiable
    with respect to each shard's unscaled bf16 logits (gradients in bf16)."""
    if len(logits) != len(part.ranges):
        raise ValueError("logits must have one entry per shard")
    logp, entropy, _ = _LinearLogpFromLogits.apply(part, y, float(tau), *logits)
    return logp, entropy


class _Embedding(torch.autograd.Function):
    @staticmethod
    def forward(ctx, ids, part, scale, out_dtype, *W):
        y = lp_embedding(ids, list(W), part, scale=scale, out_dtype=out_dtype)
        ctx.part, ctx.scale = part, scale
        ctx.dtype = next(w.dtype for w in W if w is not None)
        ctx.save_for_backward(ids)
        return y

    @staticmethod
    @once_differentiable
    def backward(ctx, g):
        (ids,) = ctx.saved_tensors
        # a gradient that was broadcast or transposed has rows the library does not take
        if g.stride(1) != 1 or (g.stride(0) * g.element_size()) % 16 != 0 or g.data_ptr() % 16 != 0 \
                or g.stride(0) < g.shape[1]:
            g = g.clone(memory_format=torch.contiguous_format)
        dW = lp_embedding_backward(ids, g, ctx.part, scale=ctx.scale, dw_dtype=ctx.dtype)
        return (None, None, None, None, *[d if ctx.needs_input_grad[4 + k] else None for k, d in enumerate(dW)])


def embedding(ids: torch.Tensor, W: Sequence[torch.Tensor], part, scale: float = 1.0, out_dtype=None):
    """Embedding lookup with autograd: scale * W[ids] (see lp_embedding), differentiable with
    respect to every W[k]; the gradients have the table's type. For a table that is tied to
    the head and trained with fp32 gradients, call lp_embedding_backward with accumulate=True on
    the dW of lp_backward_ex instead: that adds the two without rounding either."""
    return _Embedding.apply(ids, part, float(scale), out_dtype, *W)


def _check_options(function, options):
    """Refuses the options of the library call that the wrapper gives itself."""
    for name in ("upstream", "grads", "metrics"):
        if name in options:
            raise TypeError(f"{name} is not an option of {function} under autograd, which sets it")


def _save(ctx, inputs, options):
    """Keeps the inputs and the tensors among the options with autograd, which notices when one was changed in
    place before the backward reads it again."""
    ctx.names = [k for k, v in options.items() if isinstance(v, torch.Tensor) and k != "workspace"]
    ctx.options = {k: v for k, v in options.items() if k not in ctx.names}
    ctx.save_for_backward(*inputs, *[options[k] for k in ctx.names])


def _saved(ctx, n):
    """The n inputs, and the options, that _save kept."""
    saved = ctx.saved_tensors
    return saved[:n], {**ctx.options, **dict(zip(ctx.names, saved[n:]))}


class _PolicyLoss(torch.autograd.Function):
    @staticmethod
    def forward(ctx, logp, entropy, old_logp, advantages, options):
        out = lp_policy_loss(logp, old_logp, advantages, entropy=entropy, grads=False, **options)
        _save(ctx, (logp, entropy, old_logp, advantages), options)
        ctx.mark_non_differentiable(out["metrics"], out["counts"])
        return out["metrics"][0].clone(), out["metrics"], out["counts"]

    @staticmethod
    @once_differentiable
    def backward(ctx, g, _g_metrics, _g_counts):
        (logp, entropy, old_logp, advantages), options = _saved(ctx, 4)
        out = lp_policy_loss(logp, old_logp, advantages, entropy=entropy, metrics=False,
                             upstream=g.to(torch.float32), **options)
        return (out["grad_logp"] if ctx.needs_input_grad[0] else None,
                out["grad_entropy"] if ctx.needs_input_grad[1] else None, None, None, None)


def policy_loss(logp: torch.Tensor, old_logp: torch.Tensor, advantages: torch.Tensor,
                entropy: Optional[torch.Tensor] = None, **options):
    """lp_policy_loss with autograd: returns (loss, metrics, counts), the loss differentiable with
    respect to logp and entropy. ``options`` are those of lp_policy_loss (ref_logp, mask, cu_seqlens,
    clip_low, clip_high, dual_clip, kl_coef, kl_kind, entropy_coef, aggregation, denominator,
    adv_per_seq, workspace). The backward is one library call that reads the inputs again and multiplies by
    the upstream gradient where it is."""
    _check_options("policy_loss", options)
    return _PolicyLoss.apply(logp, entropy, old_logp, advantages, options)


class _PreferenceLoss(torch.autograd.Function):
    @staticmethod
    def forward(ctx, logp, cu_seqlens, options):
        out = lp_preference_loss(logp, cu_seqlens, grads=False, **options)
        _save(ctx, (logp, cu_seqlens), options)
        ctx.mark_non_differentiable(out["metrics"], out["counts"], out["margins"])
        return out["metrics"][0].clone(), out["metrics"], out["counts"], out["margins"]

    @staticmethod
    @once_differentiable
    def backward(ctx, g, _g_metrics, _g_counts, _g_margins):
        (logp, cu_seqlens), options = _saved(ctx, 2)
        out = lp_preference_loss(logp, cu_seqlens, metrics=False, upstream=g.to(torch.float32), **options)
        return out["grad_logp"], None, None


def preference_loss(logp: torch.Tensor, cu_seqlens: torch.Tensor, **options):
    """lp_preference_loss with autograd: returns (loss, metrics, counts, margins), the loss
    differentiable with respect to logp. ``options`` are those of lp_preference_loss (ref_logp,
    mask, beta, kind, label_smoothing, length_normalised, margin, denominator, workspace)."""
    _check_options("preference_loss", options)
    return _PreferenceLoss.apply(logp, cu_seqlens, options)
