"""Plain 64-bit definitions of the residual norm, its gradient, dropout and the balance loss, in elementary torch
operations on whatever device the inputs are, with bounds of what fp32 arithmetic may differ by."""
import torch

U = 2.0 ** -24
HALF_STEP = {torch.bfloat16: 2.0 ** -8, torch.float32: U}


# ------------------------------------------------------------------ dropout

def philox(counter, key):
    """Philox4x32-10 on Python integers: four counter words, two key words."""
    c, k = list(counter), list(key)
    for _ in range(10):
        p, q = c[0] * 0xD2511F53, c[2] * 0xCD9E8D57
        c = [(q >> 32) ^ c[1] ^ k[0], q & 0xFFFFFFFF, (p >> 32) ^ c[3] ^ k[1], p & 0xFFFFFFFF]
        k = [(k[0] + 0x9E3779B9) & 0xFFFFFFFF, (k[1] + 0xBB67AE85) & 0xFFFFFFFF]
    return c


def _multiply(x, m):
    """(high, low) words of x * m for words x held in int64 (the product of two words would pass 2^63)."""
    high, low = (x >> 16) * m, (x & 0xFFFF) * m
    total = ((high & 0xFFFF) << 16) + low
    return (high >> 16) + (total >> 32), total & 0xFFFFFFFF


def kept(T, H, p, seed, offset=0, row_start=0, device="cpu"):
    """Which elements of [T, H] are kept, and the factor of those."""
    seed, offset, M = seed % (1 << 64), offset % (1 << 64), 0xFFFFFFFF
    n = (torch.arange(T, device=device)[:, None] + row_start) * (H // 8) + torch.arange(H // 8, device=device)
    c = [n & M, n >> 32, torch.full_like(n, offset & M), torch.full_like(n, offset >> 32)]
    k = [seed & M, seed >> 32]
    for _ in range(10):
        (ph, pl), (qh, ql) = _multiply(c[0], 0xD2511F53), _multiply(c[2], 0xCD9E8D57)
        c = [qh ^ c[1] ^ k[0], ql, ph ^ c[3] ^ k[1], pl]
        k = [(k[0] + 0x9E3779B9) & M, (k[1] + 0xBB67AE85) & M]
    bits = torch.stack([h for w in c for h in (w & 0xFFFF, w >> 16)], dim=2).reshape(T, H)
    threshold = round(p * 65536)
    return bits >= threshold, (65536 / (65536 - threshold) if threshold < 65536 else 0.0)


def dropped(x, p, seed, offset=0, row_start=0):
    keep, factor = kept(x.shape[0], x.shape[1], p, seed, offset, row_start, x.device)
    return torch.where(keep, x.double() * factor, 0.0)


# ------------------------------------------------------------------ residual norm

def _wide(w, like, offset):
    return torch.ones(like.shape[1], dtype=torch.float64, device=like.device) if w is None else w.double() + offset


def _rms(x, eps):
    return (x.square().mean(1, keepdim=True) + eps).rsqrt()


# A sum of a row in fp32 has at most 16 additions in a thread, 5 over lanes and 16 over warps, and two CTAs: 64 U
# relative to the sum of magnitudes, with the products. A root of it has half of that, and what is multiplied by
# it a few roundings more.
ROW = 64 * U


def norm(h, y=None, weight=None, post_norm=False, post_weight=None, gate=None, residual_scale=1.0, eps=1e-6,
         weight_offset=0.0, dropout=0.0, seed=0, offset=0, row_start=0):
    """(h_out, norm) and what fp32 may differ by in each, before they are rounded to their types."""
    u = h.double()
    tol = torch.zeros_like(u)
    if y is not None:
        b = y.double()
        if post_norm:
            b = b * _rms(b, eps) * _wide(post_weight, b, weight_offset)
        if gate is not None:
            b = b * (gate.double() if gate.dim() != 1 else gate.double()[None])
        if dropout:
            keep, factor = kept(*b.shape, dropout, seed, offset, row_start, b.device)
            b = torch.where(keep, b * factor, 0.0)
        tol = ROW * (b.abs() + (residual_scale * u).abs())
        u = residual_scale * u + b
    r, w = _rms(u, eps), _wide(weight, u, weight_offset)
    n = u * r * w
    # the mean of squares takes the errors of its terms along
    moved = r * r * (u.abs() * tol).mean(1, keepdim=True)
    return u, n, tol, (r * w).abs() * tol + n.abs() * (ROW + moved)


def norm_backward(u, y, dn, dh, weight=None, post_norm=False, post_weight=None, gate=None, residual_scale=1.0, eps=1e-6,
                  weight_offset=0.0, dropout=0.0, seed=0, offset=0, row_start=0):
    """The gradients by the formulas, each as (value, what fp32 may differ by before it is rounded)."""
    u = u.double()
    T = u.shape[0]
    D, tol = torch.zeros_like(u), torch.zeros_like(u)
    out = {}
    if dh is not None:
        D = D + dh.double()
        tol = tol + 4 * U * dh.double().abs()
    r = _rms(u, eps)
    if dn is not None:
        dn = dn.double()
        a = dn * _wide(weight, u, weight_offset)
        au, abs_au = (a * u).mean(1, keepdim=True), (a * u).abs().mean(1, keepdim=True)
        D = D + r * a - u * r ** 3 * au
        tol = tol + 2 * ROW * ((r * a).abs() + u.abs() * r ** 3 * (abs_au + au.abs()))
        x = dn * u * r
        out["d_weight"] = (x.sum(0), (2 * ROW + T * U) * x.abs().sum(0))
    out["d_h"] = (residual_scale * D, abs(residual_scale) * (tol + 4 * U * D.abs()))
    if y is None:
        return out
    y = y.double()
    if dropout:
        keep, factor = kept(*u.shape, dropout, seed, offset, row_start, u.device)
        D, tol, y_at = torch.where(keep, D * factor, 0.0), torch.where(keep, tol * factor, 0.0), torch.where(keep, y, 0.0)
    else:
        y_at = y
    tol = tol + 4 * U * D.abs()
    q = _rms(y, eps) if post_norm else torch.ones_like(y[:, :1])
    wp = _wide(post_weight if post_norm else None, y, weight_offset)
    g = torch.ones_like(y) if gate is None else gate.double().expand_as(y) if gate.dim() != 1 else gate.double()[None].expand_as(y)
    if dropout and gate is not None and gate.shape == y.shape:
        g = torch.where(keep, g, 0.0)
    b = y_at * q * wp
    x, tx = D * b, tol * b.abs() + ROW * (D * b).abs()
    if gate is not None:
        if gate.dim() == 1:
            out["d_gate"] = (x.sum(0), tx.sum(0) + T * U * x.abs().sum(0))
        elif gate.shape[1] == 1 and y.shape[1] != 1:
            out["d_gate"] = (x.sum(1, keepdim=True), tx.sum(1, keepdim=True) + ROW * x.abs().sum(1, keepdim=True))
        else:
            out["d_gate"] = (x, tx)
    e, te = D * g, tol * g.abs() + 4 * U * (D * g).abs()
    if post_norm:
        x = e * y_at * q
        out["d_post_weight"] = (x.sum(0), (te * (y_at * q).abs() + ROW * x.abs()).sum(0) + T * U * x.abs().sum(0))
        a, ta = e * wp, te * wp.abs() + 4 * U * (e * wp).abs()
        s, abs_s = (a * y).mean(1, keepdim=True), (a * y).abs().mean(1, keepdim=True)
        ts = (ta * y.abs()).mean(1, keepdim=True) + ROW * abs_s
        out["d_y"] = (q * a - y * q ** 3 * s,
                      q * ta + 2 * ROW * (q * a).abs() + y.abs() * q ** 3 * (ts + 2 * ROW * s.abs()))
    else:
        out["d_y"] = (e, te)
    return out


# ------------------------------------------------------------------ balance loss

def balance(logits, ids, coef=1.0, z_coef=0.0, score="softmax", mask=None, cu=None):
    """(metrics, expert counts, counts, gradient) and what fp32 may differ by in metrics and gradient."""
    dev = logits.device
    T, E = logits.shape
    K = ids.shape[1]
    keep = torch.ones(T, dtype=torch.bool, device=dev) if mask is None else mask != 0
    l = torch.where(keep[:, None], logits.double(), 0.0)
    if cu is None:
        seg, S = torch.zeros(T, dtype=torch.int64, device=dev), 1
    else:
        S = cu.numel() - 1
        seg = torch.repeat_interleave(torch.arange(S, device=dev), cu.long().diff())
    n = torch.zeros(S, dtype=torch.int64, device=dev).index_add_(0, seg, keep.long())
    used = keep[:, None] & (ids >= 0)
    at = (seg[:, None] * E + ids.long())[used]
    c = torch.zeros(S * E, dtype=torch.int64, device=dev).index_add_(0, at, torch.ones_like(at)).reshape(S, E)
    f = (c * E).double() / (K * n.clamp(min=1)).double()[:, None] - 1.0     # less one, exactly where c E = K n
    f_tol = 4 * U * (f.abs() + U)
    N, seqs = int(keep.sum()), int((n > 0).sum())
    if score == "softmax":
        top = l.max(1, keepdim=True).values
        top = torch.where(top == -float("inf"), 0.0, top)
        q = torch.exp(l - top)
        total = q.sum(1, keepdim=True)
        p = torch.where(total > 0, q / total, 0.0)
        lse = torch.where(total[:, 0] > 0, (top + total.log())[:, 0], 0.0)
        # an exponent (the difference to the top, in units of log 2) is rounded twice, its power twice over
        scale = 1 + (l - top).abs().clamp(max=200.0)
        v = torch.ones_like(p)
    else:
        q = torch.sigmoid(l)
        small = q.sum(1, keepdim=True) < 1e-20
        top = l.max(1, keepdim=True).values
        top = torch.where(top == -float("inf"), 0.0, top)
        q = torch.where(small, torch.exp(l - top), q)
        total = q.sum(1, keepdim=True)
        p = torch.where(total > 0, q / total, 0.0)
        lse = torch.zeros(T, dtype=torch.float64, device=dev)
        scale = 1 + torch.where(small, l - top, l).abs().clamp(max=200.0)
        v = torch.where(small, 1.0, torch.sigmoid(-l))
    rel = 12 * U * scale
    p_tol = p * (rel + (p * rel).sum(1, keepdim=True) + 32 * U) + 1e-30
    fs, fs_tol = f[seg], f_tol[seg]
    d = (fs * p).sum(1, keepdim=True)
    d_tol = (p_tol * fs.abs() + p * fs_tol).sum(1, keepdim=True) + 32 * U * (fs * p).abs().sum(1, keepdim=True)
    w = torch.where(keep, 1.0 / (n[seg].clamp(min=1) * max(seqs, 1)).double(), 0.0)[:, None]
    whole = (p.sum(1, keepdim=True) > 0).double()
    lse_tol = 16 * U * (1 + lse.abs()) + (p * rel).sum(1)
    grad = coef * w * p * (fs - d) * v
    tol = abs(coef) * w * v * (p_tol * (fs - d).abs() + p * (fs_tol + d_tol) + (16 * U + rel) * p * (fs - d).abs())
    zw = z_coef * 2 * torch.where(keep, lse, 0.0)[:, None] / max(N, 1)
    grad = grad + zw * p
    tol = tol + (zw * p_tol).abs() + 8 * U * (zw * p).abs() \
        + abs(z_coef) * 2 * torch.where(keep, lse_tol, 0.0)[:, None] / max(N, 1) * p
    # the kernel adds the two terms' factors first: f a + (z - a d)
    tol = tol + 8 * U * p * (zw.abs() + abs(coef) * w * v * (fs.abs() + d.abs()))
    b, b_tol = (w * (d + whole)).sum(), (w * (d_tol + 64 * U * (d.abs() + 1))).sum()
    zk = torch.where(keep, lse, 0.0)
    z = (zk ** 2).sum() / max(N, 1)
    z_tol = (2 * zk.abs() * torch.where(keep, lse_tol, 0.0)).sum() / max(N, 1) + 64 * U * z
    load = float(c.sum(0).max()) * E / (K * N) if N else 0.0
    b_tol, z_tol = b_tol + T * U * b.abs() / 64, z_tol + T * U * z / 64
    metrics = torch.stack([coef * b + z_coef * z, b, z, torch.tensor(load, dtype=torch.float64, device=dev)])
    m_tol = torch.stack([abs(coef) * b_tol + abs(z_coef) * z_tol + 4 * U * metrics[0].abs(), b_tol, z_tol,
                         torch.tensor(8 * U * load, dtype=torch.float64, device=dev)])
    counts = torch.tensor([N, 0 if cu is None else seqs], device=dev)
    return metrics, c.sum(0), counts, grad, m_tol, tol
