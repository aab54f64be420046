"""fp64 CPU oracle of the embedding, the policy loss and the preference loss.

TEST INFRASTRUCTURE ONLY, like the package it sits in: plain numpy in float64, written from the
definitions in include/lp.h, sharing no code with the library. Loops over sequences and tokens are
meant: they follow the definitions term by term. policy_loss_of_long and preference_loss_of_long are the
same functions over whole arrays, for batches of millions of tokens.
"""
from __future__ import annotations

import math

import numpy as np


def embedding(ids, W, vocab_start, scale):
    """W: fp64 [V, H], rows vocab_start, vocab_start + 1, ...; ids outside them give zero rows."""
    out = np.zeros((len(ids), W.shape[1]))
    for t, v in enumerate(ids):
        if vocab_start <= v < vocab_start + W.shape[0]:
            out[t] = scale * W[v - vocab_start]
    return out


def embedding_backward(ids, dY, vocab_start, width, scale, dW=None):
    """(dW, sum of |scale dY| per element, positions per row); dW is added to when given."""
    H = dY.shape[1]
    total, mag, n = np.zeros((width, H)), np.zeros((width, H)), np.zeros(width, dtype=np.int64)
    for t, v in enumerate(ids):
        r = v - vocab_start
        if v >= 0 and 0 <= r < width:
            total[r] += scale * dY[t]
            mag[r] += abs(scale) * np.abs(dY[t])
            n[r] += 1
    return (total if dW is None else dW + total), mag, n


def _weights(mask, cu, aggregation, denominator):
    T = len(mask)
    kept = [int(np.count_nonzero(mask[a:b])) for a, b in zip(cu[:-1], cu[1:])]
    seqs, tokens = sum(n > 0 for n in kept), int(np.count_nonzero(mask))
    w = np.zeros(T)
    if aggregation == "token_mean":
        den = denominator if denominator > 0 else tokens
        if den > 0:
            w[mask] = 1.0 / den
    else:
        den = denominator if denominator > 0 else seqs
        for i, (a, b) in enumerate(zip(cu[:-1], cu[1:])):
            if kept[i]:
                per = kept[i] if aggregation == "seq_mean_token_mean" else 1
                w[a:b] = np.where(mask[a:b], 1.0 / (per * den), 0.0)
    return w, tokens, seqs


def policy_loss(logp, old, adv, ref=None, entropy=None, mask=None, cu=None, clip_low=0.2, clip_high=0.2, dual=0.0,
                kl_coef=0.0, kl="k3", entropy_coef=0.0, aggregation="token_mean", denominator=0.0, per_seq=False):
    """dict: metrics [6], counts (tokens, sequences), grad_logp, grad_entropy, and `mag`, the sum over
    tokens of the magnitude of each metric's terms."""
    T = len(logp)
    mask = np.ones(T, dtype=bool) if mask is None else np.asarray(mask) != 0
    has_seqs = cu is not None
    cu = [0, T] if cu is None else [int(x) for x in cu]
    w, tokens, seqs = _weights(mask, cu, aggregation, denominator)
    terms = np.zeros((5, T))
    g, ge = np.zeros(T), np.zeros(T)
    seq = np.repeat(np.arange(len(cu) - 1), np.diff(cu))
    for t in np.nonzero(mask)[0]:
        A = float(adv[seq[t]] if per_seq else adv[t])
        r = math.exp(float(logp[t]) - float(old[t]))
        loss, slope, clipped = -r * A, -r * A, False
        for hit, bound in ((A > 0 and r > 1 + clip_high, 1 + clip_high), (A < 0 and r < 1 - clip_low, 1 - clip_low),
                           (dual and A < 0 and r > dual, dual)):
            if hit:
                loss, slope, clipped = -bound * A, 0.0, True
        k = dk = 0.0
        if ref is not None:
            x = float(ref[t]) - float(logp[t])
            k, dk = {"k1": (-x, 1.0), "k2": (x * x / 2, -x), "k3": (math.expm1(x) - x, -math.expm1(x))}[kl]
        e = float(entropy[t]) if entropy is not None else 0.0
        terms[:, t] = w[t] * np.array([loss, k, e, clipped, r])
        g[t] = w[t] * (slope + (kl_coef * dk if kl_coef else 0.0))
        ge[t] = -w[t] * entropy_coef
    m, mag = terms.sum(axis=1), np.abs(terms).sum(axis=1)
    total = m[0] + kl_coef * m[1] - entropy_coef * m[2]
    mag0 = mag[0] + abs(kl_coef) * mag[1] + abs(entropy_coef) * mag[2]
    return {"metrics": np.concatenate([[total], m]), "mag": np.concatenate([[mag0], mag]),
            "counts": (tokens, seqs if has_seqs else 0), "grad_logp": g, "grad_entropy": ge, "weights": w}


def preference_loss(logp, cu, ref=None, mask=None, beta=0.1, kind="sigmoid", smoothing=0.0, normalised=False,
                    margin=0.0, denominator=0.0):
    """dict: metrics [5], count, margins, grad_logp, `slopes` (d loss / d h per pair, before the mean)."""
    T, P = len(logp), (len(cu) - 1) // 2
    cu = [int(x) for x in cu]
    mask = np.ones(T, dtype=bool) if mask is None else np.asarray(mask) != 0
    s, n = np.zeros(2 * P), np.zeros(2 * P, dtype=np.int64)
    mag = np.zeros(2 * P)
    for i in range(2 * P):
        x = [float(logp[t]) - (float(ref[t]) if ref is not None else 0.0) for t in range(cu[i], cu[i + 1]) if mask[t]]
        n[i] = len(x)
        if n[i]:
            per = n[i] if normalised else 1
            s[i], mag[i] = math.fsum(x) / per, math.fsum(abs(v) for v in x) / per
    counted = [p for p in range(P) if n[2 * p] and n[2 * p + 1]]
    den = denominator if denominator > 0 else len(counted)
    h, slopes, g = np.zeros(P), np.zeros(P), np.zeros(T)
    m = np.zeros(5)
    for p in counted:
        h[p] = s[2 * p] - s[2 * p + 1] - margin
        x = beta * h[p]
        if kind == "sigmoid":
            loss = (1 - smoothing) * np.logaddexp(0, -x) + smoothing * np.logaddexp(0, x)
            slopes[p] = beta * (smoothing * np.exp(-np.logaddexp(0, -x)) - (1 - smoothing) * np.exp(-np.logaddexp(0, x)))
        elif kind == "hinge":
            loss, slopes[p] = max(0.0, 1 - x), -beta if x < 1 else 0.0
        else:
            loss, slopes[p] = (h[p] - 1 / (2 * beta)) ** 2, 2 * (h[p] - 1 / (2 * beta))
        m += np.array([loss, h[p] > 0, x, beta * s[2 * p], beta * s[2 * p + 1]]) / den
        for i, sign in ((2 * p, 1.0), (2 * p + 1, -1.0)):
            per = n[i] if normalised else 1
            for t in range(cu[i], cu[i + 1]):
                if mask[t]:
                    g[t] = sign * slopes[p] / den / per
    return {"metrics": m, "count": len(counted), "margins": h, "grad_logp": g, "slopes": slopes, "mag": mag}


def _kept(mask, cu):
    """Kept tokens of each sequence."""
    before = np.concatenate([[0], np.cumsum(mask)])
    return (before[cu[1:]] - before[cu[:-1]]).astype(np.int64)


def policy_loss_of_long(logp, old, adv, ref=None, entropy=None, mask=None, cu=None, clip_low=0.2, clip_high=0.2, dual=0.0,
                        kl_coef=0.0, kl="k3", entropy_coef=0.0, aggregation="token_mean", denominator=0.0, per_seq=False):
    """policy_loss over whole arrays."""
    T = len(logp)
    mask = np.ones(T, dtype=bool) if mask is None else np.asarray(mask) != 0
    bounds = np.array([0, T] if cu is None else cu, dtype=np.int64)
    kept, seq = _kept(mask, bounds), np.repeat(np.arange(len(bounds) - 1), np.diff(bounds))
    tokens, seqs = int(mask.sum()), int((kept > 0).sum())
    den = denominator if denominator > 0 else max(tokens if aggregation == "token_mean" else seqs, 1)
    per = np.maximum(kept, 1)[seq] if aggregation == "seq_mean_token_mean" else 1
    w = np.where(mask, 1.0 / (den * np.float64(per)), 0.0)
    value = lambda a: np.where(mask, a, 0.0).astype(np.float64)  # noqa: E731
    A = value(np.asarray(adv)[seq] if per_seq else adv)
    r = np.exp(value(logp) - value(old))
    low, high = (A < 0) & (r < 1 - clip_low), (A > 0) & (r > 1 + clip_high)
    over = (A < 0) & (r > dual) if dual else np.zeros(T, dtype=bool)
    clipped = low | high | over
    used = np.select([low, high, over], [1 - clip_low, 1 + clip_high, dual], r)
    x = value(ref) - value(logp) if ref is not None else np.zeros(T)
    k, dk = {"k1": (-x, np.ones(T)), "k2": (x * x / 2, -x), "k3": (np.expm1(x) - x, -np.expm1(x))}[kl]
    if ref is None:
        k = dk = np.zeros(T)
    e = value(entropy) if entropy is not None else np.zeros(T)
    terms = w * np.stack([-used * A, k, e, clipped.astype(np.float64), r])
    m, mag = terms.sum(axis=1), np.abs(terms).sum(axis=1)
    total = m[0] + kl_coef * m[1] - entropy_coef * m[2]
    mag0 = mag[0] + abs(kl_coef) * mag[1] + abs(entropy_coef) * mag[2]
    return {"metrics": np.concatenate([[total], m]), "mag": np.concatenate([[mag0], mag]),
            "counts": (tokens, seqs if cu is not None else 0), "grad_logp": w * (np.where(clipped, 0.0, -r * A) + kl_coef * dk),
            "grad_entropy": -w * entropy_coef, "weights": w}


def preference_loss_of_long(logp, cu, ref=None, mask=None, beta=0.1, kind="sigmoid", smoothing=0.0, normalised=False,
                            margin=0.0, denominator=0.0):
    """preference_loss over whole arrays."""
    T, cu = len(logp), np.asarray(cu, dtype=np.int64)
    mask = np.ones(T, dtype=bool) if mask is None else np.asarray(mask) != 0
    kept, n_seqs = _kept(mask, cu), len(cu) - 1
    seq = np.repeat(np.arange(n_seqs), np.diff(cu))
    x = np.where(mask, logp, 0.0).astype(np.float64)
    if ref is not None:
        x = x - np.where(mask, ref, 0.0)
    per = np.maximum(kept, 1) if normalised else np.ones(n_seqs)
    s = np.bincount(seq, weights=x, minlength=n_seqs) / per
    mag = np.bincount(seq, weights=np.abs(x), minlength=n_seqs) / per
    counted = (kept[0::2] > 0) & (kept[1::2] > 0)
    n = int(counted.sum())
    den = denominator if denominator > 0 else max(n, 1)
    h = np.where(counted, s[0::2] - s[1::2] - margin, 0.0)
    z = beta * h
    if kind == "sigmoid":
        loss = (1 - smoothing) * np.logaddexp(0, -z) + smoothing * np.logaddexp(0, z)
        slope = beta * (smoothing * np.exp(-np.logaddexp(0, -z)) - (1 - smoothing) * np.exp(-np.logaddexp(0, z)))
    elif kind == "hinge":
        loss, slope = np.maximum(0.0, 1 - z), np.where(z < 1, -beta, 0.0)
    else:
        loss, slope = (h - 1 / (2 * beta)) ** 2, 2 * (h - 1 / (2 * beta))
    slope = np.where(counted, slope, 0.0)
    values = (loss, h > 0, z, beta * s[0::2], beta * s[1::2])
    m = np.array([float(np.sum(np.where(counted, v, 0.0))) / den for v in values])
    each = np.stack([slope, -slope], axis=1).reshape(-1) / den / per
    return {"metrics": m, "count": n, "margins": h, "grad_logp": np.where(mask, each[seq], 0.0), "slopes": slope,
            "mag": mag}
