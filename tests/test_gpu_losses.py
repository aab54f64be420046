"""lp_policy_loss and lp_preference_loss on the GPU against the fp64 oracle.

Tolerances, with u = 2^-24 (half a step of fp32). Policy: a token's ratio carries the rounding of
its exponent, |d| u, the exponential's 2 steps (4 u) and a handful of products, so its gradient is
within w u (|r A| (|d| + 12) + kl_coef e^|x| (|x| + 12)); a metric is within 128 u of the sum of its
terms' magnitudes. Preference: a sequence's sum is within 16 u of the sum of magnitudes (8 adds a lane, 5
levels of a tree, one rounding a token), a margin within that of both answers, and a slope or loss
follows by its Lipschitz constant. Inputs keep 1e-5 away from the kinks."""
import numpy as np
import pytest

from lp_util import dev_f32, dev_i32
from oracle import train

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
AGG = ("token_mean", "seq_mean_token_mean", "seq_mean_token_sum")


@pytest.fixture(scope="module")
def lp():
    from lm_head_linear_tcgen05_gb300 import _build
    _build.build()
    import lm_head_linear_tcgen05_gb300 as mod
    import torch
    assert mod.lp_device_supported()
    torch.cuda.set_device(0)
    return mod


LENGTHS = {
    "one": [1], "few": [3, 0, 1, 7], "ragged": [300, 0, 1, 513, 2, 255, 256, 257, 90], "long": [9000, 5, 4096, 0, 4097, 1],
    "empty_ends": [0, 0, 40, 0, 0], "many": [1, 2, 0, 3] * 500, "tiles": [256, 256, 1024, 4096, 0, 512], "crowded": [3, 0, 1, 2] * 700, "over": [16385, 0, 3, 40],
}


def _offsets(lengths):
    return np.concatenate([[0], np.cumsum(lengths)]).astype(np.int64)


def _tokens(lengths, seed, drop=True):
    """logp, old, ref, entropy, mask; what the mask drops is NaN or infinite."""
    rs = np.random.RandomState(seed)
    cu = _offsets(lengths)
    T = int(cu[-1])
    logp = -rs.rand(T) * 4
    d = 0.3 * rs.randn(T)
    for kink in (np.log(1.28), np.log(0.8), np.log(1.5)):
        near = np.abs(np.exp(d) - np.exp(kink)) < 1e-4
        d[near] += 1e-3
    logp = logp.astype(np.float32).astype(np.float64)
    old = (logp - d).astype(np.float32)
    ref = (logp + 0.6 * rs.randn(T)).astype(np.float32)
    mask = rs.rand(T) < 0.7
    for i in range(len(lengths)):
        if rs.rand() < 0.15:
            mask[cu[i]:cu[i + 1]] = False
    ent = (rs.rand(T) * 3).astype(np.float32)
    logp = logp.astype(np.float32)
    if drop:
        junk = np.array([np.nan, np.inf, -np.inf, 1e38], dtype=np.float32)
        for a in (logp, old, ref, ent):
            a[~mask] = junk[rs.randint(0, 4, int((~mask).sum()))]
    return cu, logp, old, ref, ent, mask, rs


@pytest.mark.parametrize("lengths", list(LENGTHS))
@pytest.mark.parametrize("aggregation", AGG)
@pytest.mark.parametrize("kl", ["k1", "k2", "k3", None])
@pytest.mark.parametrize("per_seq", [False, True])
def test_policy(lp, lengths, aggregation, kl, per_seq):
    cu, logp, old, ref, ent, mask, rs = _tokens(LENGTHS[lengths], 11)
    T, S = len(logp), len(cu) - 1
    adv = (rs.randn(S if per_seq else T) * 2).astype(np.float32)
    adv[rs.rand(len(adv)) < 0.1] = 0.0
    dual = 1.5 if kl in ("k1", "k3") else 0.0
    kc = 0.05 if kl else 0.0
    want = train.policy_loss(logp, old, adv, ref=ref if kl else None, entropy=ent, mask=mask, cu=cu, clip_low=0.2,
                             clip_high=0.28, dual=dual, kl_coef=kc, kl=kl or "k3", entropy_coef=0.01,
                             aggregation=aggregation, per_seq=per_seq)
    args = dict(ref_logp=dev_f32(ref) if kl else None, entropy=dev_f32(ent), mask=dev_u8(mask), cu_seqlens=dev_i32(cu),
                clip_low=0.2, clip_high=0.28, dual_clip=dual, kl_coef=kc, kl_kind=kl or "k3", entropy_coef=0.01,
                aggregation=aggregation, adv_per_seq=per_seq)
    out = lp.lp_policy_loss(dev_f32(logp), dev_f32(old), dev_f32(adv), **args)
    assert tuple(out["counts"].tolist()) == want["counts"]
    m = out["metrics"].double().cpu().numpy()
    assert np.all(np.abs(m - want["metrics"]) <= 128 * U * want["mag"] + 1e-30)
    A = np.where(mask, np.repeat(adv, np.diff(cu)) if per_seq else adv, 0.0)
    d = np.abs(np.where(mask, logp, 0.0) - np.where(mask, old, 0.0))
    x = np.abs(np.where(mask, ref, 0.0) - np.where(mask, logp, 0.0)) if kl else np.zeros(T)
    bound = want["weights"] * U * (np.abs(np.exp(d) * A) * (d + 12) + kc * np.exp(x) * (x + 12))
    g = out["grad_logp"].double().cpu().numpy()
    assert np.all(np.abs(g - want["grad_logp"]) <= bound + 1e-38) and np.all(g[~mask] == 0)
    ge = out["grad_entropy"].double().cpu().numpy()
    assert np.all(np.abs(ge - want["grad_entropy"]) <= 4 * U * np.abs(want["grad_entropy"]) + 1e-38)
    again = lp.lp_policy_loss(dev_f32(logp), dev_f32(old), dev_f32(adv), **args)
    for k in ("metrics", "counts", "grad_logp", "grad_entropy"):
        assert again[k].equal(out[k]), k
    assert lp.lp_get_device_error() == 0


def dev_u8(mask):
    import torch
    return torch.from_numpy(np.ascontiguousarray(mask).astype(np.uint8)).cuda()


def test_policy_without_sequences_or_mask(lp):
    import torch
    cu, logp, old, ref, ent, _, rs = _tokens([70001], 4, drop=False)
    adv = rs.randn(70001).astype(np.float32)
    want = train.policy_loss(logp, old, adv, clip_high=0.28)
    out = lp.lp_policy_loss(dev_f32(logp), dev_f32(old), dev_f32(adv), clip_high=0.28)
    assert np.all(np.abs(out["metrics"].double().cpu().numpy() - want["metrics"]) <= 128 * U * want["mag"])
    assert tuple(out["counts"].tolist()) == (70001, 0) and out["grad_entropy"] is None
    # arrays that start off a 16-byte boundary give the same bits
    shifted = [torch.cat([torch.zeros(1, device="cuda"), dev_f32(a)])[1:] for a in (logp, old, adv)]
    mask = torch.ones(70004, dtype=torch.bool, device="cuda")[3:]
    off = lp.lp_policy_loss(*shifted, mask=mask, clip_high=0.28)
    assert torch.equal(off["metrics"], out["metrics"]) and torch.equal(off["grad_logp"], out["grad_logp"])
    # the given denominator, an upstream gradient, and gradients or metrics alone
    scaled = lp.lp_policy_loss(dev_f32(logp), dev_f32(old), dev_f32(adv), clip_high=0.28, denominator=140002.0,
                               upstream=torch.tensor([4.0], device="cuda"))
    assert torch.allclose(scaled["grad_logp"], 2 * out["grad_logp"], rtol=8 * U, atol=0)
    assert abs(float(scaled["loss"]) - float(out["loss"]) / 2) <= 128 * U * want["mag"][0]
    alone = lp.lp_policy_loss(dev_f32(logp), dev_f32(old), dev_f32(adv), clip_high=0.28, metrics=False)
    assert alone["metrics"] is None and torch.equal(alone["grad_logp"], out["grad_logp"])
    alone = lp.lp_policy_loss(dev_f32(logp), dev_f32(old), dev_f32(adv), clip_high=0.28, grads=False)
    assert alone["grad_logp"] is None and torch.equal(alone["metrics"], out["metrics"])
    assert lp.lp_get_device_error() == 0


@pytest.mark.parametrize("aggregation", AGG)
def test_policy_masks_that_leave_nothing(lp, aggregation):
    import torch
    nan = torch.full((600,), float("nan"), device="cuda")
    out = lp.lp_policy_loss(nan, nan, nan, ref_logp=nan, entropy=nan, mask=torch.zeros(600, dtype=torch.bool, device="cuda"),
                            cu_seqlens=dev_i32([0, 10, 10, 600]), kl_coef=0.1, entropy_coef=0.1, aggregation=aggregation)
    assert torch.count_nonzero(out["metrics"]) == 0 and out["counts"].tolist() == [0, 0]
    assert torch.count_nonzero(out["grad_logp"]) == 0 and torch.count_nonzero(out["grad_entropy"]) == 0
    empty = torch.zeros(0, device="cuda")
    out = lp.lp_policy_loss(empty, empty, empty, aggregation=aggregation, cu_seqlens=dev_i32([0, 0]))
    assert torch.count_nonzero(out["metrics"]) == 0 and out["grad_logp"].shape == (0,)
    # a kept NaN reaches the loss and its own gradient only
    one = torch.zeros(600, device="cuda")
    bad = one.clone()
    bad[7] = float("nan")
    out = lp.lp_policy_loss(bad, one, one + 1, cu_seqlens=dev_i32([0, 10, 10, 600]), aggregation=aggregation)
    assert bool(out["loss"].isnan()) and int(out["grad_logp"].isnan().sum()) == 1
    # extreme ratios: e^200 overflows; a positive advantage clips it, the dual clip bounds a negative one
    far = torch.full((4,), 200.0, device="cuda")
    A = torch.tensor([1.0, -1.0, 1.0, -1.0], device="cuda")
    out = lp.lp_policy_loss(far, one[:4].contiguous(), A, dual_clip=3.0)
    assert abs(float(out["loss"]) - (3.0 - 1.2) / 2) < 1e-6 and torch.count_nonzero(out["grad_logp"]) == 0
    assert lp.lp_get_device_error() == 0


@pytest.mark.parametrize("cu", [[0, 5, 3, 20], [1, 5, 9, 20], [0, 5, 9, 19], [0, 5, 9, 21], [0, -7, 9, 20],
                                [0, 2 ** 31 - 1, 9, 20], [20, 9, 5, 0], [0, 0, 0, 0]])
def test_wrong_offsets_fail_closed(lp, cu):
    import torch
    x = -torch.rand(20, device="cuda")
    out = lp.lp_policy_loss(x, x, x, cu_seqlens=dev_i32(cu), aggregation="seq_mean_token_mean")
    assert lp.lp_get_device_error() == 12
    assert bool(out["metrics"].isnan().all()) and torch.count_nonzero(out["grad_logp"]) == 0
    out = lp.lp_preference_loss(x, dev_i32(cu + cu[-1:]))
    assert lp.lp_get_device_error() == 12
    assert bool(out["metrics"].isnan().all()) and torch.count_nonzero(out["grad_logp"]) == 0


def _pairs(lengths):
    return lengths if len(lengths) % 2 == 0 else list(lengths) + [3]


@pytest.mark.parametrize("lengths", list(LENGTHS))
@pytest.mark.parametrize("kind,smoothing", [("sigmoid", 0.0), ("sigmoid", 0.15), ("hinge", 0.0), ("ipo", 0.0)])
@pytest.mark.parametrize("normalised", [False, True])
@pytest.mark.parametrize("with_ref", [False, True])
def test_preference(lp, lengths, kind, smoothing, normalised, with_ref):
    cu, logp, _, ref, _, mask, _ = _tokens(_pairs(LENGTHS[lengths]), 21)
    beta, margin = 0.3, 0.125
    want = train.preference_loss(logp, cu, ref=ref if with_ref else None, mask=mask, beta=beta, kind=kind,
                                 smoothing=smoothing, normalised=normalised, margin=margin)
    assert kind != "hinge" or np.all(np.abs(beta * want["margins"] - 1) > 1e-4)
    args = dict(ref_logp=dev_f32(ref) if with_ref else None, mask=dev_u8(mask), beta=beta, kind=kind,
                label_smoothing=smoothing, length_normalised=normalised, margin=margin)
    out = lp.lp_preference_loss(dev_f32(logp), dev_i32(cu), **args)
    P, n = len(want["margins"]), want["count"]
    assert int(out["counts"][0]) == n
    seq_err = 16 * U * want["mag"]
    h, herr = want["margins"], seq_err[0::2] + seq_err[1::2] + 2 * U * (np.abs(want["margins"]) + margin)
    got = out["margins"].double().cpu().numpy()
    assert np.all(np.abs(got - h) <= herr + 1e-38)
    x, gap = np.abs(beta * h), np.abs(h) + 1 / (2 * beta)
    lip = {"sigmoid": beta * beta / 4, "hinge": 0.0, "ipo": 2.0}[kind]
    slope_err = lip * herr + U * ((x + 16) * beta if kind != "ipo" else 16 * gap)
    loss_err = beta * herr + 16 * U * (1 + x) if kind != "ipo" else 2 * gap * herr + herr ** 2 + 16 * U * gap ** 2
    den = max(n, 1)
    kept = np.array([np.count_nonzero(mask[a:b]) for a, b in zip(cu[:-1], cu[1:])])
    per = np.maximum(kept, 1) if normalised else np.ones(2 * P)
    bound = np.repeat(np.repeat(slope_err, 2) / per, np.diff(cu)) / den + 4 * U * np.abs(want["grad_logp"])
    g = out["grad_logp"].double().cpu().numpy()
    assert np.all(np.abs(g - want["grad_logp"]) <= bound + 1e-38) and np.all(g[~mask] == 0)
    m, mm = out["metrics"].double().cpu().numpy(), np.abs(want["metrics"])
    errs = [loss_err.sum(), 0.0, beta * herr.sum(), beta * seq_err[0::2].sum(), beta * seq_err[1::2].sum()]
    for i in range(5):
        # and 4 u of the terms: beta and its products, the final rounding
        terms = mm[i] + (beta * (want["mag"][0::2] + want["mag"][1::2]).sum() / den if i >= 2 else 0.0)
        assert abs(m[i] - want["metrics"][i]) <= errs[i] / den + 4 * U * terms + 1e-38, i
    again = lp.lp_preference_loss(dev_f32(logp), dev_i32(cu), **args)
    for k in ("metrics", "counts", "margins", "grad_logp"):
        assert again[k].equal(out[k]), k
    assert lp.lp_get_device_error() == 0


@pytest.mark.parametrize("lengths", [[70001, 66000], [5, 90000, 300, 0, 140000, 257], [2] * 9000 + [70000, 4]])
def test_long_and_crowded_sequences(lp, lengths):
    """Sequences of more tiles than eight lanes add, beside short ones, and tiles of many sequences."""
    cu, logp, old, ref, _, mask, rs = _tokens(lengths, 31)
    want = train.preference_loss(logp, cu, ref=ref, mask=mask, beta=0.01)
    out = lp.lp_preference_loss(dev_f32(logp), dev_i32(cu), ref_logp=dev_f32(ref), mask=dev_u8(mask), beta=0.01)
    herr = 16 * U * (want["mag"][0::2] + want["mag"][1::2]) + 2 * U * np.abs(want["margins"])
    assert np.all(np.abs(out["margins"].double().cpu().numpy() - want["margins"]) <= herr + 1e-38)
    assert int(out["counts"][0]) == want["count"]
    adv = rs.randn(len(lengths)).astype(np.float32)
    want = train.policy_loss(logp, old, adv, mask=mask, cu=cu, aggregation="seq_mean_token_mean", per_seq=True)
    out = lp.lp_policy_loss(dev_f32(logp), dev_f32(old), dev_f32(adv), mask=dev_u8(mask), cu_seqlens=dev_i32(cu),
                            aggregation="seq_mean_token_mean")
    assert tuple(out["counts"].tolist()) == want["counts"]
    assert np.all(np.abs(out["metrics"].double().cpu().numpy() - want["metrics"]) <= 128 * U * want["mag"] + 1e-30)
    assert lp.lp_get_device_error() == 0


def test_preference_extremes_and_options(lp):
    import torch
    cu = dev_i32([0, 1, 2, 3, 4])
    inf = float("inf")
    out = lp.lp_preference_loss(dev_f32([500.0, -500.0, -500.0, 500.0]), cu, beta=2.0)
    assert abs(float(out["loss"]) - 1000.0) < 1e-3 and out["metrics"][1] == 0.5
    assert torch.equal(out["grad_logp"], dev_f32([0.0, 0.0, -1.0, 1.0]))
    out = lp.lp_preference_loss(dev_f32([inf, 0.0, -1.0, -1.0]), cu)
    assert abs(float(out["loss"]) - np.log(2) / 2) < 1e-6 and not bool(out["grad_logp"].isnan().any())
    out = lp.lp_preference_loss(dev_f32([float("nan"), 0.0, -1.0, -1.0]), cu)
    assert bool(out["loss"].isnan()) and out["grad_logp"].isnan().tolist() == [True, True, False, False]
    x, ref = -torch.rand(4, device="cuda"), -torch.rand(4, device="cuda")
    base = lp.lp_preference_loss(x, cu, ref_logp=ref)
    up = lp.lp_preference_loss(x, cu, ref_logp=ref, denominator=1.0, upstream=torch.tensor(0.5, device="cuda"))
    assert torch.allclose(up["grad_logp"], base["grad_logp"], rtol=8 * U)
    assert abs(float(up["loss"]) - 2 * float(base["loss"])) < 1e-6
    empty = torch.zeros(0, device="cuda")
    out = lp.lp_preference_loss(empty, dev_i32([0, 0, 0]))
    assert torch.count_nonzero(out["metrics"]) == 0 and out["margins"].tolist() == [0.0]
    assert lp.lp_get_device_error() == 0


def test_gradients_are_the_difference_quotient(lp):
    """The loss along the sign of its gradient, by central differences of step e: they are off by e^2
    times a third derivative of order one, and by the rounding of the loss, 4 u / e."""
    import torch
    cu, logp, old, ref, _, _, rs = _tokens([200, 31, 64, 5], 2, drop=False)
    adv = dev_f32(rs.randn(300))
    logp, old, ref, cu = dev_f32(logp), dev_f32(old), dev_f32(ref), dev_i32(cu)
    e = 2.0 ** -7

    def policy(l):
        return lp.lp_policy_loss(l, old, adv, ref_logp=ref, clip_low=1.0, clip_high=50.0, kl_coef=0.5, cu_seqlens=cu,
                                 aggregation="seq_mean_token_mean")

    def preference(l):
        return lp.lp_preference_loss(l, cu, ref_logp=ref, beta=0.2, length_normalised=True)

    for f in (policy, preference):
        g = f(logp)["grad_logp"].double()
        d = g.sign().float()
        slope = (float(f(logp + e * d)["loss"]) - float(f(logp - e * d)["loss"])) / (2 * e)
        assert abs(slope - float(g.abs().sum())) <= 8 * e * e * (1 + float(g.abs().sum())) + 8 * U / e


def test_streams_and_graph(lp):
    import torch
    cu, logp, old, ref, _, _, rs = _tokens(LENGTHS["ragged"] + [7], 2, drop=False)
    logp, old, ref, cu = dev_f32(logp), dev_f32(old), dev_f32(ref), dev_i32(cu)
    adv = dev_f32(rs.randn(len(logp)))

    def both():
        a = lp.lp_policy_loss(logp, old, adv, ref_logp=ref, kl_coef=0.1, cu_seqlens=cu)
        b = lp.lp_preference_loss(logp, cu, ref_logp=ref)
        return [a["metrics"], a["grad_logp"], b["metrics"], b["grad_logp"], b["margins"]]

    want = both()
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        got = both()
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = both()
    for _ in range(3):
        for t in got:
            t.fill_(9.0)
        graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, got))
