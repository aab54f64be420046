"""What the embedding and loss operators are measured on.

Four operators: the embedding lookup, its gradient, the clipped policy loss and the preference
loss (both losses with their gradients). ``run`` computes a pass in its plain form - elementary
torch operations in 32 bits, rounded once - or, with ``own``, through this package's entry points.
"""
import math

import numpy as np
import torch

own = False

AGGREGATIONS = ("token_mean", "seq_mean_token_mean", "seq_mean_token_sum")
METRICS = 6


# ------------------------------------------------------------------ cases

def listed():
    return [
        # one decode step: a batch of 64 sequences, one new token each
        dict(name="embed_decode", op="embed", T=64, H=4096, V=151936, shards=1, table="bf16", out="bf16", scale=1.0,
             unused=0.0),
        # a batch of prompts over a table in four vocabulary shards with padded ids, scaled by sqrt(H)
        dict(name="embed_prompt", op="embed", T=8192, H=4096, V=151936, shards=4, table="bf16", out="bf16",
             scale=64.0, unused=0.02),
        # fp32 master weights, odd sizes
        dict(name="embed_fp32_odd", op="embed", T=5001, H=1032, V=128257, shards=2, table="f32", out="f32",
             scale=0.5, unused=0.1),
        # the gradient of a tiny batch: what a call costs
        dict(name="embed_grad_tiny", op="embed_grad", T=64, H=256, V=1000, shards=1, grad="bf16", dw="f32",
             scale=1.0, unused=0.0, micro=1, hot=0.0),
        # a training step's gradient over the full table, written whole in fp32
        dict(name="embed_grad_step", op="embed_grad", T=4096, H=4096, V=151936, shards=1, grad="bf16", dw="f32",
             scale=64.0, unused=0.05, micro=1, hot=0.0),
        # two micro-batches accumulated into one fp32 gradient of a small table: most rows are touched
        dict(name="embed_grad_micro", op="embed_grad", T=16384, H=2048, V=32768, shards=4, grad="bf16", dw="f32",
             scale=1.0, unused=0.05, micro=2, hot=0.05),
        # long packed batch where a few ids (padding, newline) hold most tokens; bf16 gradient
        dict(name="embed_grad_hot", op="embed_grad", T=65537, H=1024, V=32749, shards=1, grad="f32", dw="bf16",
             scale=32.0, unused=0.0, micro=1, hot=0.7),
        # one micro-batch of a policy update, no reference policy
        dict(name="policy_micro", op="policy", T=4096, S=8, agg="token_mean", kl="k3", kl_coef=0.0, ent_coef=0.0,
             dual=0.0, per_seq=False),
        # grouped responses, one advantage per response, KL and entropy terms, sequence means
        dict(name="policy_groups", op="policy", T=98304, S=64, agg="seq_mean_token_mean", kl="k3", kl_coef=0.001,
             ent_coef=0.001, dual=3.0, per_seq=True),
        # all tokens of one rank's update
        dict(name="policy_rank", op="policy", T=4194304, S=1024, agg="token_mean", kl="k3", kl_coef=0.001,
             ent_coef=0.001, dual=0.0, per_seq=False),
        # eight pairs of answers
        dict(name="preference_micro", op="preference", T=4099, P=8, kind="sigmoid", beta=0.1, smoothing=0.0,
             normalised=False, ref=True),
        # a rank's batch of pairs, smoothed labels
        dict(name="preference_rank", op="preference", T=2097143, P=1024, kind="sigmoid", beta=0.1, smoothing=0.1,
             normalised=False, ref=True),
    ]


def _log_int(rng, lo, hi):
    """An integer spread over the logarithm of its range; the large round ones are left to the listed cases."""
    n = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    return n - 1 if n > 1024 and n % 1024 == 0 else n


def _width(rng, hi):
    """A hidden size: a power of two or an odd multiple of 8."""
    if rng.random() < 0.4:
        return 1 << rng.randint(6, hi.bit_length() - 1)
    return 8 * (2 * _log_int(rng, 4, hi // 16 - 1) + 1)


def draw(rng):
    op = rng.choice(("embed", "embed_grad", "policy", "preference"))
    if op == "embed":
        return dict(op=op, T=_log_int(rng, 1, 16384), H=_width(rng, 8192), V=_log_int(rng, 1000, 151936),
                    shards=rng.choice((1, 2, 4, 8)), table=rng.choice(("bf16", "bf16", "f32")),
                    out=rng.choice(("bf16", "f32")), scale=rng.choice((1.0, 0.5, 45.25)),
                    unused=rng.choice((0.0, 0.1)))
    if op == "embed_grad":
        H = _width(rng, 4096)
        V = _log_int(rng, 1000, min(151936, 500000000 // H))
        dw = rng.choice(("f32", "f32", "bf16"))
        return dict(op=op, T=_log_int(rng, 1, min(65537, 32000000 // H)), H=H, V=V,
                    shards=rng.choice((1, 2, 4, 8)), grad=rng.choice(("bf16", "bf16", "f32")), dw=dw,
                    scale=rng.choice((1.0, 0.5, 45.25)), unused=rng.choice((0.0, 0.1)),
                    micro=rng.choice((1, 2)) if dw == "f32" else 1, hot=rng.choice((0.0, 0.0, 0.3, 0.95)))
    if op == "policy":
        T = _log_int(rng, 1, 4000000)
        ref = rng.random() < 0.7
        return dict(op=op, T=T, S=_log_int(rng, 1, max(1, min(4096, T // 2))), agg=rng.choice(AGGREGATIONS),
                    kl=rng.choice(("k1", "k2", "k3")), kl_coef=0.01 if ref else 0.0,
                    ent_coef=rng.choice((0.0, 0.001)), dual=rng.choice((0.0, 3.0)), per_seq=rng.random() < 0.5)
    T = _log_int(rng, 2, 2000000)
    return dict(op=op, T=T, P=_log_int(rng, 1, max(1, min(2048, T // 4))), kind=rng.choice(("sigmoid", "hinge", "ipo")),
                beta=rng.choice((0.1, 0.5)), smoothing=rng.choice((0.0, 0.1)), normalised=rng.random() < 0.5,
                ref=rng.random() < 0.8)


# ------------------------------------------------------------------ inputs

_DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def _ranges(c):
    """Equal shards of the vocabulary padded to a multiple of 128 * shards (none padded when whole)."""
    V, n = c["V"], c["shards"]
    padded = V if n == 1 else -(-V // (128 * n)) * 128 * n
    step = padded // n
    return V, padded, tuple((k * step, (k + 1) * step) for k in range(n))


def _ids(c, T, gen):
    """Token ids: ranks of a Zipf-like law spread over the vocabulary, a share `hot` of one id, a share
    `unused` of -1."""
    V = c["V"]
    u = torch.rand(T, device="cuda", generator=gen, dtype=torch.float64)
    rank = torch.clamp((float(V + 1) ** u).long() - 1, 0, V - 1)
    ids = (rank * 7919 + 11) % V
    pick = torch.rand(T, device="cuda", generator=gen)
    ids = torch.where(pick < c.get("hot", 0.0), V // 3, ids)
    return torch.where(pick >= 1.0 - c["unused"], -1, ids).to(torch.int32)


def _normal(shape, gen, dtype, std=1.0):
    return torch.empty(shape, dtype=dtype, device="cuda").normal_(0.0, std, generator=gen)


def _lengths(T, n, rs):
    """n sequence lengths that add up to T: lognormal, now and then an empty one."""
    w = np.exp(0.6 * rs.randn(n)) * (rs.rand(n) >= 0.02)
    if w.sum() == 0:
        w[0] = 1.0
    cu = np.floor(np.concatenate([[0.0], np.cumsum(w)]) / w.sum() * T + 0.5).astype(np.int64)
    cu[-1] = T
    return cu


def _batch(T, n, seed, gen):
    """Packed sequences: offsets, the kept tokens (each sequence begins with a prompt; some sequences are
    dropped whole) and log probabilities, -inf in some of the places that are not kept."""
    rs = np.random.RandomState(seed % (1 << 31))
    cu = _lengths(T, n, rs)
    keep = np.ones(T, dtype=np.uint8)
    if n > 1 or T > 8:
        for a, b, prompt, gone in zip(cu[:-1], cu[1:], rs.rand(n) * 0.4, rs.rand(n) < 0.03):
            keep[a:b if gone else a + int((b - a) * prompt)] = 0
    mask = torch.from_numpy(keep).cuda()
    logp = torch.log(torch.rand(T, device="cuda", generator=gen) * 0.999 + 0.001)
    dead = (mask == 0) & (torch.rand(T, device="cuda", generator=gen) < 0.1)
    logp = torch.where(dead, -math.inf, logp)
    return torch.from_numpy(cu.astype(np.int32)).cuda(), mask, logp


def prepare(case, seed):
    c = case
    gen = torch.Generator(device="cuda")
    gen.manual_seed(int(seed))
    s = {"case": c}
    if c["op"] in ("embed", "embed_grad"):
        real, padded, ranges = _ranges(c)
        s["partition"] = (real, padded, ranges)
        if c["op"] == "embed":
            s["ids"] = _ids(c, c["T"], gen)
            s["W"] = [_normal((b - a, c["H"]), gen, _DT[c["table"]], 0.02) for a, b in ranges]
        else:
            s["ids"] = [_ids(c, c["T"], gen) for _ in range(c["micro"])]
            s["dY"] = [_normal((c["T"], c["H"]), gen, _DT[c["grad"]]) for _ in range(c["micro"])]
    else:
        policy = c["op"] == "policy"
        n = c["S"] if policy else 2 * c["P"]
        s["cu"], s["mask"], s["logp"] = _batch(c["T"], n, seed, gen)
        T = c["T"]
        if policy:
            s["old"] = s["logp"] + _normal(T, gen, torch.float32, 0.15)
            s["adv"] = _normal(n if c["per_seq"] else T, gen, torch.float32) + 0.25
            s["ref"] = s["logp"] + _normal(T, gen, torch.float32, 0.3) if c["kl_coef"] else None
            s["entropy"] = torch.rand(T, device="cuda", generator=gen) * 3.0 if c["ent_coef"] else None
        else:
            s["ref"] = s["logp"] + _normal(T, gen, torch.float32, 0.3) if c["ref"] else None
    return s


# ------------------------------------------------------------------ one pass

CLIP_LOW, CLIP_HIGH = 0.2, 0.28


def run(state):
    return (_run_own if own else _run_plain)(state)


def _run_own(s):
    import lm_head_linear_tcgen05_gb300 as lp
    c = s["case"]
    if c["op"] == "embed":
        return lp.lp_embedding(s["ids"], s["W"], lp.VocabPartition(*s["partition"]), scale=c["scale"],
                               out_dtype=_DT[c["out"]])
    if c["op"] == "embed_grad":
        part = lp.VocabPartition(*s["partition"])
        dW = lp.lp_embedding_backward(s["ids"][0], s["dY"][0], part, scale=c["scale"], dw_dtype=_DT[c["dw"]])
        for ids, dY in zip(s["ids"][1:], s["dY"][1:]):
            lp.lp_embedding_backward(ids, dY, part, scale=c["scale"], accumulate=True, dW=dW)
        return dW
    if c["op"] == "policy":
        out = lp.lp_policy_loss(s["logp"], s["old"], s["adv"], ref_logp=s["ref"], entropy=s["entropy"], mask=s["mask"],
                                cu_seqlens=s["cu"], clip_low=CLIP_LOW, clip_high=CLIP_HIGH, dual_clip=c["dual"],
                                kl_coef=c["kl_coef"], kl_kind=c["kl"], entropy_coef=c["ent_coef"],
                                aggregation=c["agg"])
        return {k: out[k] for k in ("metrics", "counts", "grad_logp", "grad_entropy")}
    out = lp.lp_preference_loss(s["logp"], s["cu"], ref_logp=s["ref"], mask=s["mask"], beta=c["beta"], kind=c["kind"],
                                label_smoothing=c["smoothing"] if c["kind"] == "sigmoid" else 0.0,
                                length_normalised=c["normalised"])
    return {k: out[k] for k in ("metrics", "counts", "margins", "grad_logp")}


def _run_plain(s):
    plain = {"embed": _embed, "embed_grad": _embed_grad, "policy": _policy, "preference": _preference}
    return plain[s["case"]["op"]](s)


def _embed(s):
    c, (real, _, ranges) = s["case"], s["partition"]
    ids = s["ids"].long()
    if len(ranges) == 1:
        rows = s["W"][0][ids.clamp(min=0)].float() * c["scale"]
        return torch.where((ids >= 0)[:, None], rows, 0.0).to(_DT[c["out"]])
    step = ranges[0][1]
    rows = torch.zeros((c["T"], c["H"]), dtype=torch.float32, device="cuda")
    for k, W in enumerate(s["W"]):
        here = (ids >= k * step) & (ids < (k + 1) * step)
        rows = torch.where(here[:, None], W[(ids - k * step).clamp(0, step - 1)].float(), rows)
    return (rows * c["scale"]).to(_DT[c["out"]])


def _embed_grad(s):
    c, (_, padded, ranges) = s["case"], s["partition"]
    dW = torch.zeros((padded, c["H"]), dtype=torch.float32, device="cuda")
    for ids, dY in zip(s["ids"], s["dY"]):
        used = (ids >= 0)[:, None]
        dW.index_add_(0, ids.long().clamp(min=0), torch.where(used, dY.float(), 0.0))
    dW = (dW * c["scale"]).to(_DT[c["dw"]])
    return [dW[a:b] for a, b in ranges]


def _segments(s, n):
    """The sequence of every token."""
    where = torch.arange(s["case"]["T"], device="cuda", dtype=torch.int32)
    return torch.searchsorted(s["cu"][1:].contiguous(), where, right=True).clamp(max=n - 1)


def _policy(s):
    c = s["case"]
    keep = s["mask"] != 0
    seg = _segments(s, c["S"])
    count = torch.zeros(c["S"], dtype=torch.float32, device="cuda").index_add_(0, seg, keep.float())
    tokens, seqs = keep.sum(), (count > 0).sum()
    if c["agg"] == "token_mean":
        w = keep.float() / tokens.clamp(min=1)
    elif c["agg"] == "seq_mean_token_mean":
        w = keep.float() / (count[seg].clamp(min=1.0) * seqs.clamp(min=1))
    else:
        w = keep.float() / seqs.clamp(min=1)
    logp = torch.where(keep, s["logp"], 0.0)
    r = torch.exp(logp - torch.where(keep, s["old"], 0.0))
    A = s["adv"][seg] if c["per_seq"] else s["adv"]
    bound = torch.where(A > 0, 1.0 + CLIP_HIGH, 1.0 - CLIP_LOW)
    clipped = ((A > 0) & (r > bound)) | ((A < 0) & (r < bound))
    term = torch.where(clipped, bound, r)
    if c["dual"]:
        over = (A < 0) & (r > c["dual"])
        term, clipped = torch.where(over, c["dual"], term), clipped | over
    policy = -term * A
    grad = torch.where(clipped, 0.0, -r * A)
    kl = torch.zeros_like(logp)
    if c["kl_coef"]:
        x = torch.where(keep, s["ref"], 0.0) - logp
        if c["kl"] == "k1":
            kl, dkl = -x, torch.ones_like(x)
        elif c["kl"] == "k2":
            kl, dkl = 0.5 * x * x, -x
        else:
            kl, dkl = torch.expm1(x) - x, -torch.expm1(x)
        grad = grad + c["kl_coef"] * dkl
    ent = torch.where(keep, s["entropy"], 0.0) if c["ent_coef"] else torch.zeros_like(logp)
    m = torch.stack([(w * v).sum() for v in (policy, kl, ent, clipped.float(), r)])
    loss = m[0] + c["kl_coef"] * m[1] - c["ent_coef"] * m[2]
    return {"metrics": torch.cat([loss[None], m]), "counts": torch.stack([tokens, seqs]), "grad_logp": w * grad,
            "grad_entropy": -c["ent_coef"] * w if c["ent_coef"] else None}


def _preference(s):
    c = s["case"]
    P = c["P"]
    keep = s["mask"] != 0
    seg = _segments(s, 2 * P)
    count = torch.zeros(2 * P, dtype=torch.float32, device="cuda").index_add_(0, seg, keep.float())
    ratio = torch.where(keep, s["logp"] - s["ref"] if c["ref"] else s["logp"], 0.0)
    total = torch.zeros(2 * P, dtype=torch.float32, device="cuda").index_add_(0, seg, ratio)
    if c["normalised"]:
        total = total / count.clamp(min=1.0)
    counted = (count[0::2] > 0) & (count[1::2] > 0)
    pairs = counted.sum()
    sc, sr = torch.where(counted, total[0::2], 0.0), torch.where(counted, total[1::2], 0.0)
    h, beta = sc - sr, c["beta"]
    if c["kind"] == "sigmoid":
        e = c["smoothing"]
        x = beta * h
        soft = torch.log1p(torch.exp(-x.abs()))
        loss = (1 - e) * (soft - x.clamp(max=0.0)) + e * (soft + x.clamp(min=0.0))
        slope = -beta * ((1 - e) / (1 + torch.exp(x)) - e / (1 + torch.exp(-x)))
    elif c["kind"] == "hinge":
        loss, slope = (1 - beta * h).clamp(min=0.0), torch.where(beta * h < 1, -beta, 0.0)
    else:
        gap = h - 1 / (2 * beta)
        loss, slope = gap * gap, 2 * gap
    n = pairs.clamp(min=1)
    mean = lambda v: torch.where(counted, v, 0.0).sum() / n  # noqa: E731
    metrics = torch.stack([mean(v) for v in (loss, (h > 0).float(), beta * h, beta * sc, beta * sr)])
    slope = torch.where(counted, slope, 0.0) / n
    per_seq = torch.stack([slope, -slope], dim=1).reshape(-1)
    if c["normalised"]:
        per_seq = per_seq / count.clamp(min=1.0)
    return {"metrics": metrics, "counts": pairs[None], "margins": h, "grad_logp": torch.where(keep, per_seq[seg], 0.0)}


# ------------------------------------------------------------------ what a pass cannot do without

def work(case):
    c = case
    T = c["T"]
    if c["op"] == "embed":
        real = c["V"]
        rows = min(T, real)
        wb, ob = (2 if c["table"] == "bf16" else 4), (2 if c["out"] == "bf16" else 4)
        # distinct rows of T draws that are uniform in the logarithm of their rank
        distinct = min(rows, real / math.log(real + 1) * (1 + math.log(1 + T / (real / math.log(real + 1)))))
        return {"bytes": 4 * T + distinct * c["H"] * wb + T * c["H"] * ob, "flops": T * c["H"]}
    if c["op"] == "embed_grad":
        gb, db = (2 if c["grad"] == "bf16" else 4), (2 if c["dw"] == "bf16" else 4)
        used = 1.0 - c["unused"]
        return {"bytes": c["micro"] * (4 * T + used * T * c["H"] * gb) + c["V"] * c["H"] * db,
                "flops": c["micro"] * used * T * c["H"]}
    if c["op"] == "policy":
        arrays = 2 + (not c["per_seq"]) + bool(c["kl_coef"]) + bool(c["ent_coef"])
        return {"bytes": T * (4 * arrays + 1 + 4 + 4 * bool(c["ent_coef"])) + 4 * c["S"] * (1 + c["per_seq"]),
                "flops": 25 * T}
    return {"bytes": T * (4 + 4 * c["ref"] + 1 + 4) + 12 * c["P"], "flops": 4 * T}


# ------------------------------------------------------------------ the definition in 64 bits

def exact(case, seed):
    """The operators' definitions on the inputs of prepare(case, seed), in double precision."""
    c, s = case, prepare(case, seed)
    if c["op"] == "embed":
        _, padded, ranges = s["partition"]
        out = torch.zeros((c["T"], c["H"]), dtype=torch.float64, device="cuda")
        for (a, b), W in zip(ranges, s["W"]):
            at = torch.nonzero((s["ids"] >= a) & (s["ids"] < b)).reshape(-1)
            out[at] = c["scale"] * W[s["ids"][at].long() - a].double()
        return out
    if c["op"] == "embed_grad":
        _, padded, ranges = s["partition"]
        dW = torch.zeros((padded, c["H"]), dtype=torch.float64, device="cuda")
        for ids, dY in zip(s["ids"], s["dY"]):
            order = torch.argsort(ids, stable=True)
            order = order[ids[order] >= 0]
            for part in order.split(8192):
                dW.index_put_((ids[part].long(),), dY[part].double(), accumulate=True)
        return [c["scale"] * dW[a:b] for a, b in ranges]
    cu = s["cu"].cpu().numpy().astype(np.int64)
    keep = s["mask"].cpu().numpy() != 0
    f64 = lambda t: t.cpu().numpy().astype(np.float64)  # noqa: E731
    n = len(cu) - 1
    kept = np.array([int(keep[cu[i]:cu[i + 1]].sum()) for i in range(n)])
    of = np.repeat(np.arange(n), np.diff(cu))
    logp = f64(s["logp"])
    if c["op"] == "policy":
        at = np.nonzero(keep)[0]
        seqs, q = int((kept > 0).sum()), of[at]
        w = {"token_mean": np.full(len(at), 1.0 / max(1, len(at))),
             "seq_mean_token_mean": 1.0 / (np.maximum(kept, 1)[q] * max(1, seqs)),
             "seq_mean_token_sum": np.full(len(at), 1.0 / max(1, seqs))}[c["agg"]]
        r = np.exp(logp[at] - f64(s["old"])[at])
        A = f64(s["adv"])[q] if c["per_seq"] else f64(s["adv"])[at]
        hi, lo = 1.0 + CLIP_HIGH, 1.0 - CLIP_LOW
        used = np.where(A > 0, np.minimum(r, hi), np.where(A < 0, np.maximum(r, lo), r))
        if c["dual"]:
            used = np.where(A < 0, np.minimum(used, c["dual"]), used)
        moved = (used != r)
        slope = np.where(moved, 0.0, -r * A)
        kl, dkl, ent = np.zeros(len(at)), np.zeros(len(at)), np.zeros(len(at))
        if c["kl_coef"]:
            x = f64(s["ref"])[at] - logp[at]
            kl = {"k1": -x, "k2": x * x / 2, "k3": np.expm1(x) - x}[c["kl"]]
            dkl = {"k1": np.ones(len(at)), "k2": -x, "k3": -np.expm1(x)}[c["kl"]]
        if c["ent_coef"]:
            ent = f64(s["entropy"])[at]
        parts = [float(np.sum(w * v)) for v in (-used * A, kl, ent, moved, r)]
        g, ge = np.zeros(c["T"]), np.zeros(c["T"])
        g[at] = w * (slope + c["kl_coef"] * dkl)
        ge[at] = -c["ent_coef"] * w
        return {"metrics": np.array([parts[0] + c["kl_coef"] * parts[1] - c["ent_coef"] * parts[2]] + parts),
                "counts": None, "grad_logp": g, "grad_entropy": ge if c["ent_coef"] else None}
    x = np.where(keep, logp, 0.0)
    if c["ref"]:
        x = np.where(keep, x - np.where(keep, f64(s["ref"]), 0.0), 0.0)
    sums = np.array([math.fsum(x[cu[i]:cu[i + 1]]) for i in range(n)])
    scale = 1.0 / np.maximum(kept, 1) if c["normalised"] else np.ones(n)
    sums = sums * scale
    ok = (kept[0::2] > 0) & (kept[1::2] > 0)
    b, e = c["beta"], c["smoothing"]
    sc, sr = np.where(ok, sums[0::2], 0.0), np.where(ok, sums[1::2], 0.0)
    h = sc - sr
    if c["kind"] == "sigmoid":
        loss = (1 - e) * np.logaddexp(0, -b * h) + e * np.logaddexp(0, b * h)
        slope = b * (e * np.exp(-np.logaddexp(0, -b * h)) - (1 - e) * np.exp(-np.logaddexp(0, b * h)))
    elif c["kind"] == "hinge":
        loss, slope = np.maximum(0.0, 1 - b * h), np.where(b * h < 1, -b, 0.0)
    else:
        loss, slope = (h - 1 / (2 * b)) ** 2, 2 * (h - 1 / (2 * b))
    m = max(1, int(ok.sum()))
    each = np.stack([np.where(ok, slope, 0.0) / m, np.where(ok, -slope, 0.0) / m], axis=1).reshape(-1) * scale
    metrics = [float(np.sum(np.where(ok, v, 0.0))) / m for v in (loss, h > 0, b * h, b * sc, b * sr)]
    return {"metrics": np.array(metrics), "counts": None, "margins": h, "grad_logp": np.where(keep, each[of], 0.0)}
