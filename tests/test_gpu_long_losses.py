"""lp_policy_loss and lp_preference_loss where a warp takes several stretches of tokens and a CTA several groups of
pairs, against the fp64 oracle.

In the one-launch form (up to 16384 tokens) a warp takes a second stretch of 128 tokens from 8193 tokens on, a CTA a
second group of pairs from 257 answers on, and the pairs ask for more CTAs than the tokens from 33 answers on. In the
staged form that is 466945 tokens (policy), 933889 (preference), 9729 answers and 77825 sequences.

Tolerances, with u = 2^-24: those of the short batches (test_gpu_losses.py), which bound each token, sequence and pair.
A metric's partial sums are longer here: four tokens a stretch and lane, at most three stretches, then 5 and 8 adds of a
warp and a CTA, at (|d| + 12) u a term, is still below 128 u of the sum of magnitudes for |d| < 16; the CTAs' sums carry
their rounding. A pair whose h (or whose beta h - 1, for the hinge) is within its error of the kink may fall on either side."""
import numpy as np
import pytest

from lp_util import dev_f32, dev_i32
from oracle import train
from test_gpu_losses import AGG, U, _tokens, dev_u8

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def lp():
    from lm_head_linear_tcgen05_gb300 import _build
    _build.build()
    import lm_head_linear_tcgen05_gb300 as mod
    import torch
    assert mod.lp_device_supported()
    torch.cuda.set_device(0)
    return mod


def _spread(T, n, seed):
    """n lengths that add up to T, one in eight of them 0."""
    rs = np.random.RandomState(seed)
    w = rs.rand(n) * (rs.rand(n) >= 0.125)
    w[-1] += 0.5
    ends = np.floor(np.cumsum(w) / w.sum() * T + 0.5).astype(np.int64)
    ends[-1] = T
    return np.diff(np.concatenate([[0], ends])).tolist()


def _batch(lengths, seed):
    """The first of the seeds from `seed` on whose masks keep more than 0.55 of the tokens: _tokens also drops whole
    sequences, which may be nearly all of a batch of few."""
    while True:
        batch = _tokens(lengths, seed)
        if batch[5].mean() > 0.55:
            return batch
        seed += 1


CROSSING = [700, 0, 129, 4000, 1, 127, 5044, 2000]       # 12001 tokens, hardly an end on a stretch's
LENGTHS = {
    "crossing": CROSSING, "whole": [16384, 0], "stretches": [128] * 128, "hundreds": [100] * 163 + [84],
    "second_half": [8192, 1, 0, 63, 65, 128, 127, 1], "long": [300000, 0, 1, 255, 444444, 3, 255299, 1],
    "many": _spread(1000003, 12000, 1), "most": _spread(1000003, 80002, 2),
}


@pytest.mark.parametrize("lengths", list(LENGTHS))
@pytest.mark.parametrize("aggregation", AGG)
@pytest.mark.parametrize("per_seq", [False, True])
def test_policy(lp, lengths, aggregation, per_seq):
    import torch
    cu, logp, old, ref, ent, mask, rs = _batch(LENGTHS[lengths], 5)
    T, S = len(logp), len(cu) - 1
    adv = (rs.randn(S if per_seq else T) * 2).astype(np.float32)
    kl = {"token_mean": "k3", "seq_mean_token_mean": "k1", "seq_mean_token_sum": "k2"}[aggregation]
    want = train.policy_loss_of_long(logp, old, adv, ref=ref, entropy=ent, mask=mask, cu=cu, clip_high=0.28, dual=1.5,
                                     kl_coef=0.05, kl=kl, entropy_coef=0.01, aggregation=aggregation, per_seq=per_seq)
    args = dict(ref_logp=dev_f32(ref), entropy=dev_f32(ent), mask=dev_u8(mask), cu_seqlens=dev_i32(cu), clip_high=0.28,
                dual_clip=1.5, kl_coef=0.05, kl_kind=kl, entropy_coef=0.01, aggregation=aggregation, adv_per_seq=per_seq)
    out = lp.lp_policy_loss(dev_f32(logp), dev_f32(old), dev_f32(adv), **args)
    assert tuple(out["counts"].tolist()) == want["counts"]
    m = out["metrics"].double().cpu().numpy()
    assert np.all(np.abs(m - want["metrics"]) <= 128 * U * want["mag"] + 1e-30)
    A = np.where(mask, np.repeat(adv, np.diff(cu)) if per_seq else adv, 0.0)
    d = np.abs(np.where(mask, logp, 0.0) - np.where(mask, old, 0.0))
    x = np.abs(np.where(mask, ref, 0.0) - np.where(mask, logp, 0.0))
    assert d.max() < 16
    bound = want["weights"] * U * (np.abs(np.exp(d) * A) * (d + 12) + 0.05 * np.exp(x) * (x + 12))
    g = out["grad_logp"].double().cpu().numpy()
    assert np.all(np.abs(g - want["grad_logp"]) <= bound + 1e-38) and np.all(g[~mask] == 0)
    ge = out["grad_entropy"].double().cpu().numpy()
    assert np.all(np.abs(ge - want["grad_entropy"]) <= 4 * U * np.abs(want["grad_entropy"]) + 1e-38)
    # arrays off a 16-byte boundary are read and written element by element, to the same bits
    shift = lambda a: torch.cat([a[:1], a])[1:]  # noqa: E731
    for k in ("ref_logp", "entropy", "mask"):
        args[k] = shift(args[k])
    off = lp.lp_policy_loss(shift(dev_f32(logp)), shift(dev_f32(old)), dev_f32(adv), **args)
    for k in ("metrics", "counts", "grad_logp", "grad_entropy"):
        assert off[k].equal(out[k]), k
    assert lp.lp_get_device_error() == 0


PAIRS = dict(LENGTHS)
PAIRS.update({"34_answers": _spread(300, 34, 3), "258_answers": _spread(900, 258, 4), "1024_answers": _spread(2000, 1024, 5),
              "1024_of_16384": _spread(16384, 1024, 6), "crossing_pairs": [4000, 5044, 700, 129, 2000, 127, 300, 131]})


@pytest.mark.parametrize("lengths", list(PAIRS))
@pytest.mark.parametrize("kind,smoothing,normalised,with_ref", [("sigmoid", 0.15, False, True), ("sigmoid", 0.0, True, False),
                                                                ("hinge", 0.0, True, True), ("ipo", 0.0, False, True)])
def test_preference(lp, lengths, kind, smoothing, normalised, with_ref):
    cu, logp, _, ref, _, mask, _ = _batch(PAIRS[lengths], 9)
    beta, margin = 0.3, 0.125
    want = train.preference_loss_of_long(logp, cu, ref=ref if with_ref else None, mask=mask, beta=beta, kind=kind,
                                         smoothing=smoothing, normalised=normalised, margin=margin)
    out = lp.lp_preference_loss(dev_f32(logp), dev_i32(cu), ref_logp=dev_f32(ref) if with_ref else None,
                                mask=dev_u8(mask), beta=beta, kind=kind, label_smoothing=smoothing,
                                length_normalised=normalised, margin=margin)
    P, n = len(want["margins"]), max(want["count"], 1)
    assert int(out["counts"][0]) == want["count"]
    seq_err = 16 * U * want["mag"]
    h, herr = want["margins"], seq_err[0::2] + seq_err[1::2] + 2 * U * (np.abs(want["margins"]) + margin)
    assert np.all(np.abs(out["margins"].double().cpu().numpy() - h) <= herr + 1e-38)
    z, gap = np.abs(beta * h), np.abs(h) + 1 / (2 * beta)
    lip = {"sigmoid": beta * beta / 4, "hinge": 0.0, "ipo": 2.0}[kind]
    slope_err = lip * herr + U * ((z + 16) * beta if kind != "ipo" else 16 * gap)
    if kind == "hinge":
        slope_err = slope_err + np.where(np.abs(beta * h - 1) <= beta * herr + 4 * U, beta, 0.0)
    loss_err = beta * herr + 16 * U * (1 + z) if kind != "ipo" else 2 * gap * herr + herr ** 2 + 16 * U * gap ** 2
    kept = np.diff(np.concatenate([[0], np.cumsum(mask)])[cu])
    per = np.maximum(kept, 1) if normalised else np.ones(2 * P)
    bound = np.repeat(np.repeat(slope_err, 2) / per, np.diff(cu)) / n + 4 * U * np.abs(want["grad_logp"])
    g = out["grad_logp"].double().cpu().numpy()
    assert np.all(np.abs(g - want["grad_logp"]) <= bound + 1e-38) and np.all(g[~mask] == 0)
    counted = (kept[0::2] > 0) & (kept[1::2] > 0)
    m, mm = out["metrics"].double().cpu().numpy(), np.abs(want["metrics"])
    total = lambda v: float(v[counted].sum())  # noqa: E731
    errs = [total(loss_err), total((np.abs(h) <= herr).astype(float)), beta * total(herr), beta * total(seq_err[0::2]),
            beta * total(seq_err[1::2])]
    for i in range(5):
        # and 4 u of the terms: beta and its products, the final rounding
        terms = mm[i] + (beta * total(want["mag"][0::2] + want["mag"][1::2]) / n if i >= 2 else 0.0)
        assert abs(m[i] - want["metrics"][i]) <= errs[i] / n + 4 * U * terms + 1e-38, i
    assert lp.lp_get_device_error() == 0
