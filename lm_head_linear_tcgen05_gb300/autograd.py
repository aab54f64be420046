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

The operator's neighbours in a training step have wrappers of the same kind: embedding, dropout,
residual_norm, balance_loss, policy_loss and preference_loss.

    h = dropout(embedding(ids, [W], part), 0.1, seed)
    h, X = residual_norm(h, block(h), weight=norm_weight, dropout=0.1, seed=seed, offset=1)
    logp, entropy = linear_logp(X, [W], None, part, y, tau)
    loss, metrics, counts = policy_loss(logp, old_logp, advantages, entropy=entropy, entropy_coef=1e-3)
    (loss + balance_loss(router_logits, experts, coef=1e-2)[0]).backward()
"""
from __future__ import annotations

from typing import Optional, Sequence

import torch
from torch.autograd.function import once_differentiable

from . import (lp_backward_ex, lp_backward_from_logits, lp_balance_loss, lp_dropout, lp_embedding, lp_embedding_backward,
               lp_forward, lp_forward_from_logits, lp_policy_loss, lp_preference_loss, lp_residual_norm,
               lp_residual_norm_backward)


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


def _rows_taken(g: Optional[torch.Tensor]) -> Optional[torch.Tensor]:
    """A gradient of [T, H]; one that was broadcast or transposed has rows the library does not take."""
    if g is not None and (g.stride(1) != 1 or (g.stride(0) * g.element_size()) % 16 != 0 or g.data_ptr() % 16 != 0
                          or g.stride(0) < g.shape[1]):
        g = g.clone(memory_format=torch.contiguous_format)
    return g


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
        g = _rows_taken(g)
        dW = lp_embedding_backward(ids, g, ctx.part, scale=ctx.scale, dw_dtype=ctx.dtype)
        return (None, None, None, None, *[d if ctx.needs_input_grad[4 + k] else None for k, d in enumerate(dW)])


def embedding(ids: torch.Tensor, W: Sequence[torch.Tensor], part, scale: float = 1.0, out_dtype=None):
    """Embedding lookup with autograd: scale * W[ids] (see lp_embedding), differentiable with
    respect to every W[k]; the gradients have the table's type. For a table that is tied to
    the head and trained with fp32 gradients, call lp_embedding_backward with accumulate=True on
    the dW of lp_backward_ex instead: that adds the two without rounding either."""
    return _Embedding.apply(ids, part, float(scale), out_dtype, *W)


class _Dropout(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, p, seed, offset, row_start, rng):
        ctx.options = (p, seed, offset, row_start)
        ctx.save_for_backward(rng)
        return lp_dropout(x, p, seed, offset=offset, row_start=row_start, rng=rng)

    @staticmethod
    @once_differentiable
    def backward(ctx, g):
        p, seed, offset, row_start = ctx.options
        (rng,) = ctx.saved_tensors
        return (lp_dropout(_rows_taken(g), p, seed, offset=offset, row_start=row_start, rng=rng),) + (None,) * 5


def dropout(x: torch.Tensor, p: float, seed: int, offset: int = 0, row_start: int = 0,
            rng: Optional[torch.Tensor] = None) -> torch.Tensor:
    """lp_dropout with autograd. No mask is kept: the backward makes the same bits again, from ``rng`` too, which
    must not change before it has run."""
    return _Dropout.apply(x, float(p), int(seed), int(offset), int(row_start), rng)


class _ResidualNorm(torch.autograd.Function):
    @staticmethod
    def forward(ctx, h, y, weight, post_weight, gate, rng, options):
        h_out, norm = lp_residual_norm(h, y, weight=weight, post_weight=post_weight, gate=gate, rng=rng, **options)
        ctx.options = {k: v for k, v in options.items() if k not in ("norm", "norm_dtype")}
        ctx.save_for_backward(h_out, y, weight, post_weight, gate, rng)
        ctx.set_materialize_grads(False)
        return (None, norm) if y is None else (h_out, norm)

    @staticmethod
    @once_differentiable
    def backward(ctx, g_h, g_norm):
        if g_h is None and g_norm is None:
            return (None,) * 7
        h_out, y, weight, post_weight, gate, rng = ctx.saved_tensors
        _, want_y, want_w, want_wp, want_gate, _, _ = ctx.needs_input_grad
        vectors = [t for t in (weight, post_weight, gate) if t is not None and t.dim() == 1]
        r = lp_residual_norm_backward(h_out, y, _rows_taken(g_norm), _rows_taken(g_h), weight=weight,
                                      post_weight=post_weight, gate=gate, rng=rng, gate_grad=want_gate,
                                      dw_dtype=vectors[0].dtype if vectors else torch.float32,
                                      weight_grad=want_w or want_wp, **ctx.options)
        return (r["d_h"] if ctx.needs_input_grad[0] else None, r["d_y"] if want_y else None,
                r["d_weight"] if want_w else None, r["d_post_weight"] if want_wp else None, r["d_gate"], None, None)


def residual_norm(h: torch.Tensor, y: Optional[torch.Tensor] = None, weight: Optional[torch.Tensor] = None,
                  post_weight: Optional[torch.Tensor] = None, gate: Optional[torch.Tensor] = None,
                  rng: Optional[torch.Tensor] = None, **options):
    """lp_residual_norm with autograd: returns (h_out, norm), both differentiable with respect to h, y, the weights
    and the gate (without y: (h, the norm of h)). ``options`` are those of lp_residual_norm (post_norm, residual_scale,
    eps, weight_offset, dropout, seed, offset, row_start, norm, norm_dtype). The backward reads h_out, not h, and
    makes dropout's bits again. Gradients have the types of what they are of; for fp32 sums beside bf16 weights,
    or added to earlier ones, call lp_residual_norm_backward."""
    if "out" in options:
        raise TypeError("out is not an option of residual_norm under autograd, whose outputs are its own")
    h_out, norm = _ResidualNorm.apply(h, y, weight, post_weight, gate, rng, options)
    return (h if y is None else h_out), norm


class _BalanceLoss(torch.autograd.Function):
    @staticmethod
    def forward(ctx, logits, ids, options):
        out = lp_balance_loss(logits, ids, grads=False, **options)
        _save(ctx, (logits, ids), options)
        ctx.mark_non_differentiable(out["metrics"], out["expert_counts"], out["counts"])
        return out["metrics"][0].clone(), out["metrics"], out["expert_counts"], out["counts"]

    @staticmethod
    @once_differentiable
    def backward(ctx, g, _g_metrics, _g_experts, _g_counts):
        (logits, ids), options = _saved(ctx, 2)
        out = lp_balance_loss(logits, ids, metrics=False, upstream=g.to(torch.float32), **options)
        return out["grad_logits"], None, None


def balance_loss(logits: torch.Tensor, ids: torch.Tensor, **options):
    """lp_balance_loss with autograd: returns (loss, metrics, expert_counts, counts), the loss differentiable with
    respect to logits (the counts are not differentiated). ``options`` are those of lp_balance_loss (coef,
    z_coef, score, mask, cu_seqlens, workspace)."""
    _check_options("balance_loss", options, "out", "grad_dtype")
    return _BalanceLoss.apply(logits, ids, options)


def _check_options(function, options, *more):
    """Refuses the options of the library call that the wrapper gives itself."""
    for name in ("upstream", "grads", "metrics") + more:
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
