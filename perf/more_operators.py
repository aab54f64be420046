"""What the operators between the embedding and the losses are measured on.

Four operators: the norms around a block fused with its gate, residual and dropout; their gradient; dropout
alone; the balance loss of a router with its per-expert counts and gradient. ``run`` computes a pass in its
plain form - elementary torch operations in 32 bits, rounded once - or, with ``own``, through this package's
entry points.
"""
import math

import numpy as np
import torch

own = False

GATES = ("none", "channel", "token", "full")
EPS = 1e-6


# ------------------------------------------------------------------ cases

def listed():
    return [
        # one decode step of 64 sequences: a block's output joins the stream, the next block's norm follows
        dict(name="norm_decode", op="norm", T=64, H=4096, stream="bf16", branch="bf16", y=True, post=False, gate="none",
             p=0.0, scale=1.0, wo=0.0, pad=0),
        # a batch of prompts through a block with norms on both sides and a gate per channel
        dict(name="norm_prompt", op="norm", T=16384, H=4096, stream="bf16", branch="bf16", y=True, post=True,
             gate="channel", p=0.0, scale=1.0, wo=1.0, pad=0),
        # an fp32 stream of odd width, the block's output a slice of a wider buffer, a gate per token, dropout
        dict(name="norm_stream32_odd", op="norm", T=5001, H=1032, stream="f32", branch="bf16", y=True, post=False,
             gate="token", p=0.1, scale=1.25, wo=0.0, pad=40),
        # the norm in front of the head, no block output
        dict(name="norm_final", op="norm", T=4099, H=8192, stream="bf16", branch="bf16", y=False, post=False,
             gate="none", p=0.0, scale=1.0, wo=0.0, pad=0),
        # the gradient of a tiny batch: what a call costs
        dict(name="norm_grad_tiny", op="norm_grad", T=64, H=256, stream="bf16", branch="bf16", y=True, post=False,
             gate="none", p=0.0, scale=1.0, wo=0.0, pad=0),
        # one block of a training step: both norms, a gate per channel, dropout
        dict(name="norm_grad_step", op="norm_grad", T=8192, H=4096, stream="bf16", branch="bf16", y=True, post=True,
             gate="channel", p=0.1, scale=1.0, wo=0.0, pad=0),
        # an fp32 stream of odd width over a long batch, a gate for every element
        dict(name="norm_grad_stream32_odd", op="norm_grad", T=20001, H=1032, stream="f32", branch="bf16", y=True,
             post=False, gate="full", p=0.0, scale=0.5, wo=0.0, pad=0),
        # dropout of a few embedded prompts
        dict(name="dropout_micro", op="dropout", T=128, H=4096, dtype="bf16", p=0.1, row_start=0),
        # dropout of a long packed batch, this rank's rows of it
        dict(name="dropout_batch", op="dropout", T=65536, H=4096, dtype="bf16", p=0.05, row_start=131072),
        # a micro-batch's router, with the z term
        dict(name="balance_micro", op="balance", T=4096, E=64, K=8, S=0, dtype="f32", score="softmax", z=0.001,
             masked=0.0),
        # a layer's router over a rank's batch
        dict(name="balance_layer", op="balance", T=65536, E=128, K=8, S=0, dtype="f32", score="softmax", z=0.0,
             masked=0.05),
        # balance within each sequence, sigmoid scores in bf16
        dict(name="balance_sequences", op="balance", T=131071, E=256, K=8, S=64, dtype="bf16", score="sigmoid", z=0.0,
             masked=0.1),
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
    op = rng.choice(("norm", "norm", "norm_grad", "norm_grad", "dropout", "balance", "balance"))
    if op in ("norm", "norm_grad"):
        H = _width(rng, 16384)
        y = rng.random() < 0.85
        return dict(op=op, T=_log_int(rng, 1, min(65536, (40000000 if op == "norm" else 25000000) // H)), H=H,
                    stream=rng.choice(("bf16", "f32")), branch=rng.choice(("bf16", "bf16", "f32")), y=y,
                    post=y and rng.random() < 0.5, gate=rng.choice(GATES) if y else "none",
                    p=rng.choice((0.0, 0.1, 0.5)) if y else 0.0, scale=rng.choice((1.0, 0.5, 1.25)) if y else 1.0,
                    wo=rng.choice((0.0, 1.0)), pad=rng.choice((0, 0, 8, 136)))
    if op == "dropout":
        H = _width(rng, 16384)
        return dict(op=op, T=_log_int(rng, 1, min(262144, 120000000 // H)), H=H, dtype=rng.choice(("bf16", "f32")),
                    p=rng.choice((0.02, 0.1, 0.5, 0.9)), row_start=rng.choice((0, 5, 123456789)))
    E = _log_int(rng, 2, 512)
    T = _log_int(rng, 1, min(262144, 30000000 // E))
    score = rng.choice(("softmax", "softmax", "sigmoid"))
    return dict(op=op, T=T, E=E, K=rng.randint(1, min(8, E)),
                S=_log_int(rng, 1, max(1, min(1024, T // 2))) if rng.random() < 0.5 else 0,
                dtype=rng.choice(("f32", "f32", "bf16")), score=score,
                z=rng.choice((0.0, 0.001)) if score == "softmax" else 0.0, masked=rng.choice((0.0, 0.1)))


# ------------------------------------------------------------------ inputs

_DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def _normal(shape, gen, dtype, std=1.0, mean=0.0):
    return torch.empty(shape, dtype=dtype, device="cuda").normal_(mean, std, generator=gen)


def _lengths(T, n, rs):
    """n sequence lengths that add up to T: lognormal, now and then an empty one."""
    w = np.exp(0.6 * rs.randn(n)) * (rs.rand(n) >= 0.02)
    if w.sum() == 0:
        w[0] = 1.0
    cu = np.floor(np.concatenate([[0.0], np.cumsum(w)]) / w.sum() * T + 0.5).astype(np.int64)
    cu[-1] = T
    return cu


def prepare(case, seed):
    c = case
    gen = torch.Generator(device="cuda")
    gen.manual_seed(int(seed))
    rs = np.random.RandomState(seed % (1 << 31))
    T = c["T"]
    s = {"case": c, "seed": int(rs.randint(1, 1 << 31)) * 4294967291 % (1 << 63), "offset": int(rs.randint(0, 1 << 20))}
    if c["op"] == "dropout":
        s["x"] = _normal((T, c["H"]), gen, _DT[c["dtype"]])
        return s
    if c["op"] == "balance":
        E = c["E"]
        # popularity differs between experts; a router's logits, and the K largest of a token with a little
        # noise, as a selection bias leaves them; a few slots went unused for want of capacity
        logits = _normal((T, E), gen, torch.float32, 1.2) + _normal((E,), gen, torch.float32, 0.7)
        ids = torch.topk(logits + _normal((T, E), gen, torch.float32, 0.1), c["K"], dim=1).indices
        unused = torch.rand((T, c["K"]), device="cuda", generator=gen) < 0.01
        s["ids"] = torch.where(unused, -1, ids).to(torch.int32)
        s["logits"] = logits.to(_DT[c["dtype"]])
        s["mask"] = None
        if c["masked"]:
            s["mask"] = (torch.rand(T, device="cuda", generator=gen) >= c["masked"]).to(torch.uint8)
        s["cu"] = torch.from_numpy(_lengths(T, c["S"], rs).astype(np.int32)).cuda() if c["S"] else None
        return s
    H, stream, branch = c["H"], _DT[c["stream"]], _DT[c["branch"]]
    s["h"] = _normal((T, H), gen, stream, 2.0)
    s["y"] = _normal((T, H + c["pad"]), gen, branch, 0.5)[:, :H] if c["y"] else None
    mean = 1.0 - c["wo"]
    s["w"] = _normal((H,), gen, branch, 0.2, mean)
    s["wp"] = _normal((H,), gen, branch, 0.2, mean) if c["post"] else None
    s["gate"] = {"none": lambda: None, "channel": lambda: _normal((H,), gen, branch, 0.3, 0.5),
                 "token": lambda: torch.rand((T, 1), device="cuda", generator=gen),
                 "full": lambda: _normal((T, H), gen, branch, 0.3, 0.5)}[c["gate"]]()
    if c["op"] == "norm_grad":
        s["dn"] = _normal((T, H), gen, branch)
        s["dh"] = _normal((T, H), gen, stream)
    return s


# ------------------------------------------------------------------ one pass

def run(state):
    return (_run_own if own else _run_plain)(state)


def _run_own(s):
    import lm_head_linear_tcgen05_gb300 as lp
    c = s["case"]
    if c["op"] == "dropout":
        return lp.lp_dropout(s["x"], c["p"], s["seed"], offset=s["offset"], row_start=c["row_start"])
    if c["op"] == "balance":
        out = lp.lp_balance_loss(s["logits"], s["ids"], coef=0.01, z_coef=c["z"], score=c["score"], mask=s["mask"],
                                 cu_seqlens=s["cu"])
        return {k: out[k] for k in ("metrics", "expert_counts", "counts", "grad_logits")}
    options = dict(weight=s["w"], post_norm=c["post"], post_weight=s["wp"], gate=s["gate"], residual_scale=c["scale"],
                   eps=EPS, weight_offset=c["wo"], dropout=c["p"], seed=s["seed"], offset=s["offset"])
    if c["op"] == "norm":
        h_out, norm = lp.lp_residual_norm(s["h"], s["y"], norm_dtype=_DT[c["branch"]], **options)
        return {"h_out": h_out if c["y"] else None, "norm": norm}
    out = lp.lp_residual_norm_backward(s["h"], s["y"], s["dn"], s["dh"], **options)
    return {k: out[k] for k in ("d_h", "d_y", "d_weight", "d_post_weight", "d_gate")}


def _run_plain(s):
    plain = {"norm": _norm, "norm_grad": _norm_grad, "dropout": _dropout, "balance": _balance}
    return plain[s["case"]["op"]](s)


_LOW = 0xFFFFFFFF


def _philox(c0, c1, c2, c3, k0, k1):
    """Four words of Philox4x32-10 (Salmon, Moraes, Dror, Shaw 2011) for counters and a key of 32-bit words in
    int64; the ten rounds are the generator's definition."""
    for _ in range(10):
        a, b = c0 * 0xD2511F53, c2 * 0xCD9E8D57
        c0, c1, c2, c3 = ((b >> 32) & _LOW) ^ c1 ^ k0, b & _LOW, ((a >> 32) & _LOW) ^ c3 ^ k1, a & _LOW
        k0, k1 = (k0 + 0x9E3779B9) & _LOW, (k1 + 0xBB67AE85) & _LOW
    return torch.stack((c0, c1, c2, c3), dim=-1)


def _kept(T, H, p, seed, offset, row_start):
    """Where an element is kept. Eight neighbours of a row share a counter, 16 bits each; (1 / (1 - p), kept)."""
    drop = int(round(p * 65536))
    groups = H // 8
    g = (torch.arange(T, device="cuda")[:, None] + row_start) * groups + torch.arange(groups, device="cuda")
    hi = torch.full_like(g, offset & _LOW)
    words = _philox(g & _LOW, g >> 32, hi, torch.full_like(g, offset >> 32), seed & _LOW, seed >> 32)
    bits = torch.stack((words & 0xFFFF, words >> 16), dim=-1)
    return 65536.0 / (65536 - drop), (bits >= drop).reshape(T, H)


def _dropout(s):
    c = s["case"]
    factor, kept = _kept(c["T"], c["H"], c["p"], s["seed"], s["offset"], c["row_start"])
    return torch.where(kept, s["x"].float() * factor, 0.0).to(_DT[c["dtype"]])


def _gate(s):
    """The gate in 32 bits: [H], [T, 1] or [T, H]."""
    return 1.0 if s["gate"] is None else s["gate"].float()


def _rms(x):
    return 1.0 / torch.sqrt((x * x).mean(dim=1, keepdim=True) + EPS)


def _norm(s):
    c = s["case"]
    u = s["h"].float()
    if c["y"]:
        b = s["y"].float()
        if c["post"]:
            b = b * _rms(b) * (s["wp"].float() + c["wo"])
        b = b * _gate(s)
        if c["p"]:
            factor, kept = _kept(c["T"], c["H"], c["p"], s["seed"], s["offset"], 0)
            b = torch.where(kept, b * factor, 0.0)
        u = u * c["scale"] + b
    n = u * _rms(u) * (s["w"].float() + c["wo"])
    return {"h_out": u.to(_DT[c["stream"]]) if c["y"] else None, "norm": n.to(_DT[c["branch"]])}


def _norm_grad(s):
    c = s["case"]
    u, dn = s["h"].float(), s["dn"].float()
    r = _rms(u)
    a = dn * (s["w"].float() + c["wo"])
    D = s["dh"].float() + r * a - u * (r * r * r * (a * u).mean(dim=1, keepdim=True))
    out = {"d_h": (c["scale"] * D).to(_DT[c["stream"]]), "d_y": None, "d_weight": (dn * u * r).sum(0),
           "d_post_weight": None, "d_gate": None}
    if not c["y"]:
        return out
    if c["p"]:
        factor, kept = _kept(c["T"], c["H"], c["p"], s["seed"], s["offset"], 0)
        D = torch.where(kept, D * factor, 0.0)
    y = s["y"].float()
    ry = _rms(y) if c["post"] else 1.0
    if c["gate"] != "none":
        g = D * y * ry
        if c["post"]:
            g = g * (s["wp"].float() + c["wo"])
        out["d_gate"] = {"channel": lambda: g.sum(0), "token": lambda: g.sum(1, keepdim=True),
                         "full": lambda: g.to(_DT[c["branch"]])}[c["gate"]]()
    db = D * _gate(s)
    if c["post"]:
        out["d_post_weight"] = (db * y * ry).sum(0)
        a = db * (s["wp"].float() + c["wo"])
        db = ry * a - y * (ry * ry * ry * (a * y).mean(dim=1, keepdim=True))
    out["d_y"] = db.to(_DT[c["branch"]])
    return out


def _balance(s):
    c = s["case"]
    T, E, K, S = c["T"], c["E"], c["K"], c["S"]
    keep = torch.ones(T, dtype=torch.bool, device="cuda") if s["mask"] is None else s["mask"] != 0
    tokens = keep.sum()
    used = keep[:, None] & (s["ids"] >= 0)
    if S:
        seg = torch.searchsorted(s["cu"][1:].contiguous(), torch.arange(T, device="cuda", dtype=torch.int32),
                                 right=True).clamp(max=S - 1)
    else:
        seg = torch.zeros(T, dtype=torch.int64, device="cuda")
    n = torch.zeros(max(S, 1), dtype=torch.float32, device="cuda").index_add_(0, seg, keep.float())
    seqs = (n > 0).sum()
    where = torch.where(used, seg[:, None] * E + s["ids"], max(S, 1) * E).reshape(-1)
    count = torch.zeros(max(S, 1) * E + 1, dtype=torch.int64, device="cuda")
    count = count.index_add_(0, where, torch.ones_like(where))[:-1].reshape(-1, E)
    f = count.float() * (E / K) / n.clamp(min=1.0)[:, None]
    l = torch.where(keep[:, None], s["logits"].float(), 0.0)
    top = l.max(dim=1, keepdim=True).values
    e = torch.exp(l - top)
    total = e.sum(dim=1, keepdim=True)
    lse = (top + torch.log(total))[:, 0]
    side = 1.0
    if c["score"] == "sigmoid":
        e = 1.0 / (1.0 + torch.exp(-l))
        total = e.sum(dim=1, keepdim=True)
        side = 1.0 - e
    p = e / total
    f = f[seg]
    d = (f * p).sum(dim=1)
    w = torch.where(keep, 1.0 / (n[seg].clamp(min=1.0) * seqs.clamp(min=1)), 0.0)
    balance = (w * d).sum()
    wz = torch.where(keep, 1.0 / tokens.clamp(min=1), 0.0)
    z = (wz * lse * lse).sum() if c["score"] == "softmax" else torch.zeros_like(balance)
    grad = 0.01 * w[:, None] * p * (f - d[:, None]) * side
    if c["z"]:
        grad = grad + (c["z"] * 2.0 * wz * lse)[:, None] * p
    experts = count.sum(0)
    load = experts.max().float() * (E / K) / tokens.clamp(min=1)
    return {"metrics": torch.stack([0.01 * balance + c["z"] * z, balance, z, load]), "expert_counts": experts,
            "counts": torch.stack([tokens, seqs if S else torch.zeros_like(tokens)]),
            "grad_logits": grad.to(_DT[c["dtype"]])}


# ------------------------------------------------------------------ what a pass cannot do without

def work(case):
    c = case
    size = {"bf16": 2, "f32": 4}
    T = c["T"]
    if c["op"] == "dropout":
        return {"bytes": 2 * T * c["H"] * size[c["dtype"]], "flops": T * c["H"]}
    if c["op"] == "balance":
        return {"bytes": 2 * T * c["E"] * size[c["dtype"]] + 4 * T * c["K"] + (T if c["masked"] else 0) + 8 * c["E"],
                "flops": 8 * T * c["E"]}
    n, st, br = T * c["H"], size[c["stream"]], size[c["branch"]]
    gate = {"none": 0, "channel": c["H"] * br, "token": 4 * T, "full": n * br}[c["gate"]]
    weights = c["H"] * br * (1 + c["post"])
    if c["op"] == "norm":
        return {"bytes": n * (st + br + c["y"] * (st + br)) + gate + weights, "flops": n * (4 + 8 * c["y"])}
    d_gate = 4 * c["H"] if c["gate"] == "channel" else gate
    return {"bytes": n * (3 * st + br + c["y"] * 2 * br) + gate + d_gate + weights + 4 * c["H"] * (1 + c["post"]),
            "flops": n * (10 + 14 * c["y"])}


# ------------------------------------------------------------------ the definition in 64 bits

def _mul32(x, m):
    """(high, low) 32 bits of x * m from products of 16-bit halves."""
    x1, x0, m1, m0 = x >> 16, x & 0xFFFF, m >> 16, m & 0xFFFF
    mid = x1 * m0 + ((x0 * m0) >> 16)
    low = x0 * m1 + (mid & 0xFFFF)
    return x1 * m1 + (mid >> 16) + (low >> 16), ((low & 0xFFFF) << 16) | ((x0 * m0) & 0xFFFF)


def _kept64(T, H, p, seed, offset, row_start):
    rows = []
    for at in range(0, T, 8192):
        n = min(8192, T - at)
        index = (torch.arange(at, at + n, device="cuda").reshape(n, 1) + row_start) * (H // 8) \
            + torch.arange(H // 8, device="cuda").reshape(1, H // 8)
        x = [index % 2 ** 32, index // 2 ** 32, torch.zeros_like(index) + offset % 2 ** 32,
             torch.zeros_like(index) + offset // 2 ** 32]
        key = [seed % 2 ** 32, seed // 2 ** 32]
        for r in range(10):
            (h0, l0), (h1, l1) = _mul32(x[0], 0xD2511F53), _mul32(x[2], 0xCD9E8D57)
            x = [h1 ^ x[1] ^ ((key[0] + r * 0x9E3779B9) % 2 ** 32), l1,
                 h0 ^ x[3] ^ ((key[1] + r * 0xBB67AE85) % 2 ** 32), l0]
        halves = [v for word in x for v in (word % 65536, word // 65536)]
        rows.append((torch.stack(halves, dim=2).reshape(n, H) >= round(p * 65536)))
    return torch.cat(rows)


def exact(case, seed):
    """The operators' definitions on the inputs of prepare(case, seed), in double precision."""
    c, s = case, prepare(case, seed)
    T = c["T"]
    if c["op"] == "dropout":
        kept = _kept64(T, c["H"], c["p"], s["seed"], s["offset"], c["row_start"])
        return s["x"].double() * kept * (65536 / (65536 - round(c["p"] * 65536)))
    if c["op"] == "balance":
        return _exact_balance(c, s)
    H = c["H"]

    def branch(y, wp, gate):
        if c["post"]:
            y = y * (y.square().sum(1, keepdim=True) / H + EPS).rsqrt() * (c["wo"] + wp)
        if c["gate"] != "none":
            y = y * gate
        if c["p"]:
            kept = _kept64(T, H, c["p"], s["seed"], s["offset"], 0)
            y = y * kept * (65536 / (65536 - round(c["p"] * 65536)))
        return y

    def norm(u, w):
        return u * (u.square().sum(1, keepdim=True) / H + EPS).rsqrt() * (c["wo"] + w)

    f64 = {k: None if s[k] is None else s[k].double().requires_grad_(c["op"] == "norm_grad")
           for k in ("h", "y", "w", "wp", "gate")}
    if c["op"] == "norm":
        u = f64["h"]
        if c["y"]:
            u = c["scale"] * u + branch(f64["y"], f64["wp"], f64["gate"])
        return {"h_out": u if c["y"] else None, "norm": norm(u, f64["w"])}
    # the chain rule by automatic differentiation: first through the norm, then through the branch
    du, dw = torch.autograd.grad(norm(f64["h"], f64["w"]), (f64["h"], f64["w"]), s["dn"].double())
    du = du + s["dh"].double()
    out = {"d_h": c["scale"] * du, "d_y": None, "d_weight": dw, "d_post_weight": None, "d_gate": None}
    if c["y"]:
        of = [k for k in ("y", "wp", "gate") if f64[k] is not None]
        grads = torch.autograd.grad(branch(f64["y"], f64["wp"], f64["gate"]), [f64[k] for k in of], du)
        out.update({{"y": "d_y", "wp": "d_post_weight", "gate": "d_gate"}[k]: g for k, g in zip(of, grads)})
    return out


def _exact_balance(c, s):
    T, E, K = c["T"], c["E"], c["K"]
    logits, ids = s["logits"].double(), s["ids"].cpu().numpy()
    keep = np.ones(T, dtype=bool) if s["mask"] is None else s["mask"].cpu().numpy() != 0
    cu = s["cu"].cpu().numpy() if c["S"] else np.array([0, T])
    kept = [int(keep[a:b].sum()) for a, b in zip(cu[:-1], cu[1:])]
    counted = sum(n > 0 for n in kept)
    p = torch.softmax(logits, 1) if c["score"] == "softmax" else torch.sigmoid(logits)
    if c["score"] == "sigmoid":
        slope = 1 - p
        p = p / p.sum(1, keepdim=True)
    lse = torch.logsumexp(logits, 1).cpu().numpy()
    grad = torch.zeros_like(logits)
    total, experts = 0.0, np.zeros(E, dtype=np.int64)
    for a, b, n in zip(cu[:-1], cu[1:], kept):
        if n == 0:
            continue
        here = ids[a:b][keep[a:b]]
        load = np.bincount(here[here >= 0].reshape(-1), minlength=E)
        experts += load
        f = torch.from_numpy(load * (E / (K * n))).cuda()
        weight = torch.from_numpy(keep[a:b] / (n * counted)).cuda()
        d = p[a:b] @ f
        total += float(weight @ d)
        g = 0.01 * weight[:, None] * p[a:b] * (f[None, :] - d[:, None])
        grad[a:b] = g * slope[a:b] if c["score"] == "sigmoid" else g
    N = max(1, sum(kept))
    z = float(np.sum(np.where(keep, lse * lse, 0.0))) / N if c["score"] == "softmax" else 0.0
    if c["z"]:
        grad += torch.from_numpy(np.where(keep, c["z"] * 2 * lse / N, 0.0)).cuda()[:, None] * p
    metrics = [0.01 * total + c["z"] * z, total, z, float(experts.max()) * E / (K * N)]
    return {"metrics": np.array(metrics), "expert_counts": None, "counts": None, "grad_logits": grad}
