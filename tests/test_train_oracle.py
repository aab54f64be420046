"""The fp64 oracle of the embedding and the losses: gradients against central differences, closed
forms, and the rules for masks and empty sequences (CPU only)."""
import math

import numpy as np
import pytest

from oracle import train


def _batch(seed, lengths):
    rs = np.random.RandomState(seed)
    T = sum(lengths)
    cu = np.concatenate([[0], np.cumsum(lengths)])
    logp = -rs.rand(T) * 3
    return rs, cu, logp, logp + 0.3 * rs.randn(T), logp + 0.5 * rs.randn(T), rs.rand(T) < 0.7


@pytest.mark.parametrize("aggregation", ["token_mean", "seq_mean_token_mean", "seq_mean_token_sum"])
@pytest.mark.parametrize("kl", ["k1", "k2", "k3"])
@pytest.mark.parametrize("dual", [0.0, 1.4])
def test_policy_gradient_is_the_difference_quotient(aggregation, kl, dual):
    rs, cu, logp, old, ref, mask = _batch(3, [5, 0, 9, 1, 7])
    adv, ent = rs.randn(len(logp)) * 2, rs.rand(len(logp))
    args = dict(ref=ref, mask=mask, cu=cu, dual=dual, kl_coef=0.1, kl=kl, entropy_coef=0.05, aggregation=aggregation)

    def loss(lg, en):
        return train.policy_loss(lg, old, adv, entropy=en, **args)["metrics"][0]

    out = train.policy_loss(logp, old, adv, entropy=ent, **args)
    r = np.exp(logp - old)
    for t in range(len(logp)):
        if min(abs(r[t] - 1.2), abs(r[t] - 0.8), abs(r[t] - 1.4)) < 1e-4:
            continue                                  # a kink between the two points
        d = np.zeros(len(logp))
        d[t] = 1e-6
        assert abs((loss(logp + d, ent) - loss(logp - d, ent)) / 2e-6 - out["grad_logp"][t]) < 1e-8
        assert abs((loss(logp, ent + d) - loss(logp, ent - d)) / 2e-6 - out["grad_entropy"][t]) < 1e-8


@pytest.mark.parametrize("kind,smoothing", [("sigmoid", 0.0), ("sigmoid", 0.2), ("hinge", 0.0), ("ipo", 0.0)])
@pytest.mark.parametrize("normalised", [False, True])
def test_preference_gradient_is_the_difference_quotient(kind, smoothing, normalised):
    _, cu, logp, _, ref, mask = _batch(5, [4, 6, 3, 0, 8, 2, 5, 7])
    args = dict(ref=ref, mask=mask, beta=0.7, kind=kind, smoothing=smoothing, normalised=normalised, margin=0.3)
    out = train.preference_loss(logp, cu, **args)
    assert out["count"] == 3                          # the second pair has an empty answer
    for t in range(len(logp)):
        d = np.zeros(len(logp))
        d[t] = 1e-6
        up, down = (train.preference_loss(logp + s * d, cu, **args)["metrics"][0] for s in (1, -1))
        assert abs((up - down) / 2e-6 - out["grad_logp"][t]) < 1e-7


def test_closed_forms():
    # ratio 1 and no extra terms: the loss is minus the mean advantage, the gradient -A / N
    logp, adv = -np.arange(1.0, 6.0), np.array([1.0, -2.0, 0.5, 0.0, 3.0])
    out = train.policy_loss(logp, logp, adv)
    assert abs(out["metrics"][0] + adv.mean()) < 1e-15 and np.allclose(out["grad_logp"], -adv / 5, atol=1e-15)
    # equal answers: log 2, slope -beta / 2
    out = train.preference_loss(np.array([-1.0, -1.0]), [0, 1, 2], beta=0.4)
    assert abs(out["metrics"][0] - math.log(2)) < 1e-15 and np.allclose(out["grad_logp"], [-0.2, 0.2], atol=1e-15)
    # nothing kept
    assert train.policy_loss(logp, logp, adv, mask=np.zeros(5))["metrics"][0] == 0.0
    assert train.preference_loss(logp, [0, 2, 5], mask=np.zeros(5))["count"] == 0


def test_embedding_gradient_is_the_transpose_of_the_lookup():
    rs = np.random.RandomState(1)
    W, ids = rs.randn(11, 8), np.array([3, 3, -1, 10, 0, 14, 3])
    dY = rs.randn(7, 8)
    g, _, n = train.embedding_backward(ids, dY, 0, 11, 1.5)
    assert n[3] == 3 and n.sum() == 5                 # -1 and 14 are nobody's
    V = rs.randn(11, 8)
    assert abs((train.embedding(ids, V, 0, 1.5) * dY).sum() - (V * g).sum()) < 1e-12
    assert np.all(train.embedding(ids, W, 0, 1.5)[[2, 5]] == 0)
