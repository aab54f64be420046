"""The whole-array forms of the loss oracles give what the term-by-term ones do (CPU only)."""
import numpy as np
import pytest

from oracle import train


def _batch(seed, n):
    rs = np.random.RandomState(seed)
    lengths = rs.randint(0, 9, n) * (rs.rand(n) < 0.8)
    lengths[0] += 3
    cu = np.concatenate([[0], np.cumsum(lengths)])
    T = int(cu[-1])
    logp, old, ref, ent = -rs.rand(T) * 3, -rs.rand(T) * 3, -rs.rand(T) * 3, rs.rand(T)
    mask = rs.rand(T) < 0.7
    for a in (logp, old, ref, ent):
        a[~mask] = np.nan
    return rs, cu, T, logp, old, ref, ent, mask


def _alike(a, b, keys):
    for k in keys:
        assert np.allclose(a[k], b[k], rtol=1e-12, atol=1e-14), k


@pytest.mark.parametrize("aggregation", ["token_mean", "seq_mean_token_mean", "seq_mean_token_sum"])
@pytest.mark.parametrize("kl", ["k1", "k2", "k3", None])
@pytest.mark.parametrize("per_seq", [False, True])
def test_policy(aggregation, kl, per_seq):
    for seed in range(4):
        rs, cu, T, logp, old, ref, ent, mask = _batch(seed, 30)
        adv = rs.randn(30 if per_seq else T)
        args = dict(ref=ref if kl else None, entropy=ent, mask=mask, cu=cu, clip_high=0.28, dual=2.0 if seed % 2 else 0.0,
                    kl_coef=0.1 if kl else 0.0, kl=kl or "k3", entropy_coef=0.01, aggregation=aggregation, per_seq=per_seq,
                    denominator=7.0 if seed == 3 else 0.0)
        a, b = train.policy_loss(logp, old, adv, **args), train.policy_loss_of_long(logp, old, adv, **args)
        _alike(a, b, ("metrics", "mag", "counts", "grad_logp", "grad_entropy", "weights"))
    full = [np.nan_to_num(x) for x in (logp, old)]
    a, b = (f(*full, np.ones(T)) for f in (train.policy_loss, train.policy_loss_of_long))
    _alike(a, b, ("metrics", "counts", "grad_logp"))
    none = np.zeros(T, dtype=bool)
    a, b = (f(logp, old, np.ones(T), mask=none, cu=cu, aggregation=aggregation)
            for f in (train.policy_loss, train.policy_loss_of_long))
    _alike(a, b, ("metrics", "counts", "grad_logp"))


@pytest.mark.parametrize("kind,smoothing", [("sigmoid", 0.0), ("sigmoid", 0.2), ("hinge", 0.0), ("ipo", 0.0)])
@pytest.mark.parametrize("normalised", [False, True])
def test_preference(kind, smoothing, normalised):
    for seed in range(4):
        _, cu, T, logp, _, ref, _, mask = _batch(seed, 30)
        args = dict(ref=ref if seed % 2 else None, mask=mask, beta=0.3, kind=kind, smoothing=smoothing,
                    normalised=normalised, margin=0.1, denominator=5.0 if seed == 3 else 0.0)
        a, b = train.preference_loss(logp, cu, **args), train.preference_loss_of_long(logp, cu, **args)
        _alike(a, b, ("metrics", "count", "margins", "grad_logp", "mag", "slopes"))
