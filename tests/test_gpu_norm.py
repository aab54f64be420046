"""lp_residual_norm, its gradient and lp_dropout on the GPU against their 64-bit definitions (block_ref.py), under
bounds that count the roundings of fp32 sums and of the outputs' types."""
import random

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
import block_ref as ref  # noqa: E402

BF, F32 = torch.bfloat16, torch.float32
GATES = ("none", "channel", "token", "full")


@pytest.fixture(scope="module")
def lp():
    from lm_head_linear_tcgen05_gb300 import _build
    _build.build()
    import lm_head_linear_tcgen05_gb300 as mod
    assert mod.lp_device_supported()
    torch.cuda.set_device(0)
    return mod


def close(got, want, tol, what):
    """got, of its own type, against 64-bit values whose fp32 computation may be off by tol."""
    assert got.shape == want.shape, (what, got.shape, want.shape)
    allowed = tol + ref.HALF_STEP[got.dtype] * (want.abs() + tol) + 1e-37
    over = ((got.double() - want).abs() / allowed)
    worst = float(over.max()) if over.numel() else 0.0
    assert worst <= 1.0, (what, worst)        # NaN is not <= 1


def rows(T, H, dtype, gen, pad=0, std=1.0, mean=0.0):
    x = torch.full((T, H + pad), float("nan"), dtype=dtype, device="cuda")
    x[:, :H].normal_(mean, std, generator=gen)
    return x[:, :H]


def case(T, H, stream, branch, post, gate, seed, pad=0, wdt=None, weights=True, y=True):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    wdt = branch if wdt is None else wdt
    vec = lambda mean: torch.empty(H, dtype=wdt, device="cuda").normal_(mean, 0.3, generator=gen)  # noqa: E731
    h = rows(T, H, stream, gen, pad, 2.0)
    yy = rows(T, H, branch, gen, 2 * pad, 0.5) if y else None
    z = {"none": lambda: None, "channel": lambda: vec(0.5), "token": lambda: torch.rand((T, 1), device="cuda", generator=gen),
         "full": lambda: rows(T, H, branch, gen, pad, 0.3, 0.5)}[gate if y else "none"]()
    return h, yy, vec(1.0) if weights else None, vec(1.0) if weights and post and y else None, z, gen


SHAPES = [(1, 8), (3, 64), (2, 72), (37, 128), (6, 200), (5, 256), (7, 264), (3, 520), (9, 1032), (2, 2048), (4, 4096),
          (3, 4104), (2, 8192), (3, 8200), (2, 12296), (3, 16384), (700, 64), (1300, 264), (650, 1032), (400, 4096),
          (333, 8200), (256, 64), (257, 64), (64, 256), (65, 256), (24, 1032), (25, 1032), (20, 8192), (2500, 72), (3000, 136), (5001, 64)]


def combos():
    """Every shape with a few of the combinations of the rest; every combination with some shape."""
    rnd = random.Random(5)
    rest = [(s, b, post, g, p) for s in (BF, F32) for b in (BF, F32) for post in (False, True) for g in GATES
            for p in (0.0, 0.25)]
    rnd.shuffle(rest)
    out = []
    for i in range(max(len(rest), 4 * len(SHAPES))):
        out.append(SHAPES[i % len(SHAPES)] + rest[i % len(rest)] + (rnd.choice((0, 8, 24)),))
    return out


def options(post, gate, p, i=0):
    return dict(post_norm=post, residual_scale=(1.0, 0.5, -1.25)[i % 3], eps=(1e-6, 1e-3)[i % 2], weight_offset=(0.0, 1.0)[i % 2],
                dropout=p, seed=0x9E3779B97F4A7C15 + i, offset=(0, 5, 1 << 40)[i % 3], row_start=(0, 3, (1 << 33) + 7)[i % 3])


@pytest.mark.parametrize("i", range(len(combos())))
def test_norm_and_gradient(lp, i):
    T, H, stream, branch, post, gate, p, pad = combos()[i]
    h, y, w, wp, z, gen = case(T, H, stream, branch, post, gate, i, pad, (BF, F32)[i // 2 % 2])
    o = dict(options(post, gate, p, i), weight=w, post_weight=wp, gate=z)
    h_out, n = lp.lp_residual_norm(h, y, **o)
    u, want, tol_u, tol_n = ref.norm(h, y, **o)
    assert h_out.dtype is stream and n.dtype is branch
    close(h_out, u, tol_u, "h_out")
    close(n, want, tol_n, "norm")
    dn, dh = rows(T, H, branch, gen, pad), rows(T, H, stream, gen, 2 * pad)
    got = lp.lp_residual_norm_backward(h_out, y, dn, dh, **o)
    for k, (v, tol) in ref.norm_backward(h_out, y, dn, dh, **o).items():
        close(got[k], v, tol, k)
    assert lp.lp_get_device_error() == 0


@pytest.mark.parametrize("T,H", [(1, 8), (5, 72), (260, 256), (3, 1032), (4, 8200), (500, 4096)])
@pytest.mark.parametrize("stream,branch", [(BF, BF), (F32, BF), (BF, F32)])
@pytest.mark.parametrize("weights", [False, True])
def test_the_norm_alone(lp, T, H, stream, branch, weights):
    h, _, w, _, _, gen = case(T, H, stream, branch, False, "none", T + H, 8, y=False, weights=weights)
    o = dict(weight=w, eps=1e-5, weight_offset=1.0)
    same, n = lp.lp_residual_norm(h, norm_dtype=branch, **o)
    assert same is h
    _, want, _, tol = ref.norm(h, **o)
    close(n, want, tol, "norm")
    dn, dh = rows(T, H, branch, gen), rows(T, H, stream, gen)
    for d in (dh, None):
        got = lp.lp_residual_norm_backward(h, None, dn, d, **o)
        v = ref.norm_backward(h, None, dn, d, **o)
        close(got["d_h"], *v["d_h"], "d_h")
        if weights:
            close(got["d_weight"], *v["d_weight"], "d_weight")
        assert got["d_y"] is None and got["d_gate"] is None and (weights or got["d_weight"] is None)


@pytest.mark.parametrize("H", [64, 256, 1032, 8200])
@pytest.mark.parametrize("post,gate,p", [(False, "none", 0.0), (True, "channel", 0.2), (False, "full", 0.2), (True, "token", 0.0)])
@pytest.mark.parametrize("which", ["norm", "stream"])
def test_one_of_the_two_gradients(lp, H, post, gate, p, which):
    """d_norm or d_h_out missing: as if it were zero."""
    T = 21
    h, y, w, wp, z, gen = case(T, H, F32, BF, post, gate, H)
    o = dict(options(post, gate, p), weight=w, post_weight=wp, gate=z)
    dn = rows(T, H, BF, gen) if which == "norm" else None
    dh = rows(T, H, F32, gen) if which == "stream" else None
    got, want = lp.lp_residual_norm_backward(h, y, dn, dh, **o), ref.norm_backward(h, y, dn, dh, **o)
    assert (got["d_weight"] is None) == (dn is None)
    for k, (v, tol) in want.items():
        close(got[k], v, tol, k)
    # without the sums no workspace is needed, and the others are the same
    less = lp.lp_residual_norm_backward(h, y, dn, dh, weight_grad=False, gate_grad=gate != "channel", **o)
    assert torch.equal(less["d_h"], got["d_h"]) and torch.equal(less["d_y"], got["d_y"]) and less["d_weight"] is None
    only = lp.lp_residual_norm(h, y, norm=False, **dict(o, weight=None))
    assert only[1] is None and torch.equal(only[0], lp.lp_residual_norm(h, y, **o)[0])


@pytest.mark.parametrize("H,stream,post,gate", [(64, F32, True, "channel"), (264, BF, False, "full"), (1032, F32, True, "none")])
def test_gradient_against_differences_of_the_definition(lp, H, stream, post, gate):
    """In 64 bits, by central differences: truncation and rounding below 1e-6 of the sum of magnitudes."""
    T = 6
    h, y, w, wp, z, gen = case(T, H, stream, F32, post, gate, H + 1)
    o = dict(options(post, gate, 0.25), eps=1e-3, residual_scale=0.75)
    u, _, _, _ = ref.norm(h, y, weight=w, post_weight=wp, gate=z, **o)
    dn, dh = rows(T, H, F32, gen), rows(T, H, stream, gen)
    got = lp.lp_residual_norm_backward(u.to(stream), y, dn, dh, weight=w, post_weight=wp, gate=z, **o)
    leaves = {"d_h": h, "d_y": y, "d_weight": w, "d_post_weight": wp, "d_gate": z}
    for k, leaf in leaves.items():
        if leaf is None:
            continue
        v = torch.randn(leaf.shape, dtype=torch.float64, device="cuda", generator=gen)

        def value(step):
            at = lambda t: t.double() + step * v if t is leaf else t  # noqa: E731
            uu, nn, _, _ = ref.norm(at(h), at(y), weight=at(w), post_weight=at(wp), gate=at(z), **o)
            return float((uu * dh.double()).sum() + (nn * dn.double()).sum())

        want, size = (value(1e-4) - value(-1e-4)) / 2e-4, float((got[k].double() * v).abs().sum())
        # a bf16 stream is rounded before the gradient sees it and d_h after it: three half steps
        allowed = (3 * 2.0 ** -8 if stream is BF else 1e-5) * size + 1e-5
        assert abs(want - float((got[k].double() * v).sum())) <= allowed, k


@pytest.mark.parametrize("H", [64, 256, 520, 4104, 12296])
def test_in_place_and_rows_of_other_buffers(lp, H):
    T = 19
    h, y, w, wp, z, gen = case(T, H, BF, BF, True, "token", H, 8)
    o = dict(options(True, "token", 0.2), weight=w, post_weight=wp, gate=z)
    h_out, n = lp.lp_residual_norm(h, y, **o)
    a, b = torch.full((T + 2, H + 16), 7.0, dtype=BF, device="cuda"), torch.full((T + 2, H + 8), 7.0, dtype=BF, device="cuda")
    lp.lp_residual_norm(h, y, out=dict(h_out=a[1:-1, :H], norm=b[1:-1, :H]), **o)
    assert torch.equal(a[1:-1, :H], h_out) and torch.equal(b[1:-1, :H], n)
    for m in (a, b):                     # nothing around the rows was written
        assert bool((m[0] == 7).all() and (m[-1] == 7).all() and (m[:, H:] == 7).all())
    h2, y2 = h.clone(), y.clone()
    lp.lp_residual_norm(h2, y2, out=dict(h_out=h2, norm=y2), **o)
    assert torch.equal(h2, h_out) and torch.equal(y2, n)
    dn, dh = rows(T, H, BF, gen), rows(T, H, BF, gen)
    want = lp.lp_residual_norm_backward(h_out, y, dn, dh, **o)
    got = lp.lp_residual_norm_backward(h_out, y, dn, dh, out=dict(d_h=dh, d_y=dn), **o)
    assert got["d_h"] is dh and got["d_y"] is dn
    for k in want:
        assert torch.equal(got[k], want[k]), k
    c = torch.full((T + 2, H + 8), 7.0, dtype=BF, device="cuda")
    dn, dh = rows(T, H, BF, gen), rows(T, H, BF, gen)
    lp.lp_residual_norm_backward(h_out, y, dn, dh, out=dict(d_h=c[1:-1, :H]), **o)
    assert bool((c[0] == 7).all() and (c[-1] == 7).all() and (c[:, H:] == 7).all())


@pytest.mark.parametrize("H,stream", [(64, BF), (200, F32), (1032, BF), (4096, BF), (16384, F32)])
@pytest.mark.parametrize("post,gate", [(True, "channel"), (False, "full")])
def test_rows_stand_alone(lp, H, stream, post, gate):
    """A row's bits do not depend on the batch it is in: parts with their row_start give the whole's, and a row that
    is not finite leaves the others as they are. Two runs give the same bits, the sums over tokens too."""
    T = 330
    h, y, w, wp, z, gen = case(T, H, stream, BF, post, gate, H)
    o = dict(options(post, gate, 0.3), weight=w, post_weight=wp)
    dn, dh = rows(T, H, BF, gen), rows(T, H, stream, gen)

    def both(a, b):
        zz = z[a:b] if gate == "full" else z
        oo = dict(o, gate=zz, row_start=o["row_start"] + a)
        h_out, n = lp.lp_residual_norm(h[a:b], y[a:b], **oo)
        g = lp.lp_residual_norm_backward(h_out, y[a:b], dn[a:b], dh[a:b], **oo)
        return dict(g, h_out=h_out, norm=n)

    whole, again = both(0, T), both(0, T)
    for k in whole:
        assert whole[k] is None or torch.equal(whole[k], again[k]), k
    by_row = ["h_out", "norm", "d_h", "d_y"] + (["d_gate"] if gate == "full" else [])
    for a, b in ((0, 1), (1, 200), (200, T)):
        part = both(a, b)
        for k in by_row:
            assert torch.equal(part[k], whole[k][a:b]), (k, a, b)
    h[7, 3], y[11, 0], dn[13, 1], dh[17, H - 1] = float("nan"), float("inf"), float("inf"), float("nan")
    bad = both(0, T)
    good = torch.ones(T, dtype=torch.bool, device="cuda")
    good[[7, 11, 13, 17]] = False
    for k in by_row:
        assert torch.equal(bad[k][good], whole[k][good]), k
        assert bool(torch.isfinite(bad[k][good]).all())


@pytest.mark.parametrize("p", [0.3, 1.0])
@pytest.mark.parametrize("gate", ["none", "full"])
@pytest.mark.parametrize("H", [64, 1032])
def test_what_is_dropped_has_no_effect(lp, p, gate, H):
    """Whatever y and the gate hold where an element is dropped, infinities and NaN among it."""
    T = 9
    h, y, w, _, z, gen = case(T, H, F32, F32, False, gate, 4)
    o = dict(weight=w, gate=z, dropout=p, seed=3)
    keep, _ = ref.kept(T, H, p, 3, device="cuda")
    dn, dh = rows(T, H, F32, gen), rows(T, H, F32, gen)

    def both():
        h_out, n = lp.lp_residual_norm(h, y, **o)
        return dict(lp.lp_residual_norm_backward(h_out, y, dn, dh, **o), h_out=h_out, norm=n)

    want = both()
    y[~keep] = float("nan")
    if gate == "full":
        z[~keep] = float("inf")
    got = both()
    for k in want:
        assert want[k] is None or torch.equal(got[k], want[k]), k
    if p == 1.0:
        assert torch.equal(got["h_out"], h) and float(got["d_y"].abs().max()) == 0.0


@pytest.mark.parametrize("H", [64, 1032, 8200])
def test_rows_of_zeros_and_tiny_eps(lp, H):
    """A row of zeros has the norm 0 and finite gradients however small eps is (1 / sqrt(eps) is, cubed it need not be)."""
    T = 4
    h, y, w, wp, _, gen = case(T, H, F32, F32, True, "none", 8)
    h.zero_()
    y.zero_()
    o = dict(weight=w, post_norm=True, post_weight=wp, eps=1e-30)
    h_out, n = lp.lp_residual_norm(h, y, **o)
    assert float(h_out.abs().max()) == 0.0 and float(n.abs().max()) == 0.0
    dn, dh = rows(T, H, F32, gen, std=1e-3), rows(T, H, F32, gen)
    got = lp.lp_residual_norm_backward(h, y, dn, dh, **o)
    want = dh.double() + dn.double() * w.double() * 1e15
    close(got["d_h"], want, 8 * ref.U * want.abs(), "d_h")
    assert float(got["d_weight"].abs().max()) == 0.0 and bool(torch.isfinite(got["d_y"]).all())


def test_empty_batches(lp):
    h, y, w, wp, z, _ = case(0, 72, BF, BF, True, "channel", 1)
    h, y = torch.empty(0, 72, dtype=BF, device="cuda"), torch.empty(0, 72, dtype=BF, device="cuda")
    o = dict(weight=w, post_norm=True, post_weight=wp, gate=z)
    h_out, n = lp.lp_residual_norm(h, y, **o)
    assert h_out.shape == n.shape == (0, 72)
    got = lp.lp_residual_norm_backward(h, y, h, h, **o)
    for k in ("d_weight", "d_post_weight", "d_gate"):
        assert float(got[k].abs().max()) == 0.0
    held = {k: torch.ones(72, device="cuda") for k in ("d_weight", "d_post_weight", "d_gate")}
    lp.lp_residual_norm_backward(h, y, h, h, accumulate=True, out=held, **o)
    assert all(bool((v == 1).all()) for v in held.values())
    assert lp.lp_dropout(h, 0.5, 1).shape == (0, 72)


@pytest.mark.parametrize("H", [128, 1032])
def test_sums_added_to_earlier_ones_and_in_bf16(lp, H):
    T = 300
    h, y, w, wp, z, gen = case(T, H, BF, BF, True, "channel", 2)
    o = dict(weight=w, post_norm=True, post_weight=wp, gate=z)
    dn, dh = rows(T, H, BF, gen), rows(T, H, BF, gen)
    names = ("d_weight", "d_post_weight", "d_gate")
    one = lp.lp_residual_norm_backward(h, y, dn, dh, **o)
    held = {k: torch.randn(H, device="cuda", generator=gen) for k in names}
    want = {k: held[k] + one[k] for k in names}
    lp.lp_residual_norm_backward(h, y, dn, dh, accumulate=True, out=held, **o)
    half = lp.lp_residual_norm_backward(h, y, dn, dh, dw_dtype=BF, **o)
    for k in names:
        assert torch.equal(held[k], want[k]) and torch.equal(half[k], one[k].to(BF)), k
    with pytest.raises(ValueError):
        lp.lp_residual_norm_backward(h, y, dn, dh, accumulate=True, **o)
    with pytest.raises(lp.LPError):
        lp.lp_residual_norm_backward(h, y, dn, dh, accumulate=True, dw_dtype=BF, out={k: v.to(BF) for k, v in held.items()}, **o)


# ------------------------------------------------------------------ dropout

@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("T,H,pad", [(1, 8, 0), (3, 72, 8), (130, 264, 0), (5, 4096, 0), (1025, 1032, 24)])
@pytest.mark.parametrize("p,offset,start", [(0.1, 0, 0), (0.5, (1 << 63) + 9, 5), (0.9, 1, (1 << 44) + 1)])
def test_dropout(lp, dtype, T, H, pad, p, offset, start):
    gen = torch.Generator(device="cuda").manual_seed(T + H)
    x = rows(T, H, dtype, gen, pad)
    seed = (1 << 64) - 12345
    got = lp.lp_dropout(x, p, seed, offset=offset, row_start=start)
    keep, factor = ref.kept(T, H, p, seed, offset, start, "cuda")
    want = torch.where(keep, x.double() * factor, 0.0)
    close(got, want, 2 * ref.U * want.abs(), "dropout")
    assert bool((got[~keep] == 0).all())
    for a, b in ((0, T // 2), (T // 2, T)):
        assert torch.equal(lp.lp_dropout(x[a:b], p, seed, offset=offset, row_start=start + a), got[a:b])
    x2 = x.clone()
    x2[~keep] = float("nan")
    assert lp.lp_dropout(x2, p, seed, offset=offset, row_start=start, out=x2) is x2 and torch.equal(x2, got)
    # seed and offset from the device are added, modulo 2^64
    rng = torch.tensor([-7, 1 << 62], dtype=torch.int64, device="cuda")
    again = lp.lp_dropout(x, p, (seed + 7) % (1 << 64), offset=(offset - (1 << 62)) % (1 << 64), row_start=start, rng=rng)
    assert torch.equal(again, got)


def test_dropout_of_nothing_and_of_all(lp):
    x = torch.randn(33, 264, device="cuda")
    assert torch.equal(lp.lp_dropout(x, 0.0, 1), x)
    x[3, 4] = float("nan")
    assert float(lp.lp_dropout(x, 1.0, 1).abs().max()) == 0.0
    assert float(lp.lp_dropout(x, 1.0 - 2.0 ** -18, 1).abs().max()) == 0.0       # held as 1


def test_the_share_that_is_kept(lp):
    """2^22 elements: the count is within six standard deviations of its mean."""
    x = torch.ones(1024, 4096, device="cuda")
    for p in (0.02, 0.5, 0.9):
        n, held = x.numel(), round(p * 65536) / 65536
        kept = int((lp.lp_dropout(x, p, 77) != 0).sum())
        assert abs(kept - n * (1 - held)) < 6 * (n * held * (1 - held)) ** 0.5


# ------------------------------------------------------------------ streams, graphs, autograd

def test_a_captured_call_draws_other_bits(lp):
    T, H = 40, 1032
    h, y, w, wp, _, gen = case(T, H, F32, BF, True, "none", 6)
    rng = torch.zeros(2, dtype=torch.int64, device="cuda")
    dn, dh = rows(T, H, BF, gen), rows(T, H, F32, gen)
    o = dict(weight=w, post_norm=True, post_weight=wp, dropout=0.4, seed=11)

    def both(**kw):
        h_out, n = lp.lp_residual_norm(h, y, **o, **kw)
        return dict(lp.lp_residual_norm_backward(h_out, y, dn, dh, **o, **kw), h_out=h_out, norm=n,
                    x=lp.lp_dropout(n, 0.4, 11, **kw))

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        both(rng=rng)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            got = both(rng=rng)
    torch.cuda.current_stream().wait_stream(s)
    for step in (1, 5):
        rng[1] = step
        graph.replay()
        want = both(offset=step)
        for k, v in want.items():
            assert v is None or torch.equal(got[k], v), (k, step)


def test_two_streams_at_once(lp):
    """Calls on two streams at a time, each with its own workspace, give what they give alone."""
    cases, want = [], []
    for i, (T, H) in enumerate(((900, 4096), (1200, 1032))):
        h, y, w, wp, z, gen = case(T, H, BF, BF, True, "channel", i)
        a = (h, y, rows(T, H, BF, gen), rows(T, H, BF, gen))
        o = dict(weight=w, post_norm=True, post_weight=wp, gate=z)
        cases.append((a, o))
        want.append(lp.lp_residual_norm_backward(*a, **o))
    streams = [torch.cuda.Stream() for _ in cases]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(5):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i].append(lp.lp_residual_norm_backward(*cases[i][0], **cases[i][1]))
    torch.cuda.synchronize()
    for i in range(2):
        for r in got[i]:
            assert all(v is None or torch.equal(v, want[i][k]) for k, v in r.items())


@pytest.mark.parametrize("post,gate,p", [(False, "none", 0.0), (True, "channel", 0.2), (True, "token", 0.0), (False, "full", 0.2)])
def test_autograd(lp, post, gate, p):
    from lm_head_linear_tcgen05_gb300.autograd import dropout, residual_norm
    T, H = 23, 264
    h, y, w, wp, z, gen = case(T, H, BF, BF, post, gate, 3)
    o = dict(post_norm=post, dropout=p, seed=5, offset=6, residual_scale=0.5)
    leaves = [t for t in (h, y, w, wp, z) if t is not None]
    for t in leaves:
        t.requires_grad_()
    x = dropout(h, 0.25, 9)
    h_out, n = residual_norm(x, y, weight=w, post_weight=wp, gate=z, **o)
    g = torch.randn(H, T, dtype=BF, device="cuda", generator=gen).t()       # a transposed gradient
    grads = torch.autograd.grad((n * g).sum() + h_out.sum(), leaves)
    with torch.no_grad():
        want = lp.lp_residual_norm_backward(h_out, y, g.contiguous(), torch.ones_like(h_out), weight=w, post_weight=wp, gate=z,
                                            dw_dtype=BF, **o)
        want["d_h"] = lp.lp_dropout(want["d_h"], 0.25, 9)
    names = [k for k, t in (("d_h", h), ("d_y", y), ("d_weight", w), ("d_post_weight", wp), ("d_gate", z)) if t is not None]
    for k, got, leaf in zip(names, grads, leaves):
        assert got.dtype is leaf.dtype and got.shape == leaf.shape and torch.equal(got, want[k]), k
    # one output alone, the norm without a block, and nothing that needs a gradient
    (gy,) = torch.autograd.grad(residual_norm(h, y, weight=w, post_weight=wp, gate=z, **o)[0].float().square().sum(), (y,))
    assert bool(torch.isfinite(gy).all())
    same, n = residual_norm(h, weight=w)
    assert same is h
    gh, gw = torch.autograd.grad(n.sum() + same.sum(), (h, w))
    one = lp.lp_residual_norm_backward(h.detach(), None, torch.ones_like(n), None, weight=w.detach(), dw_dtype=BF)
    assert torch.equal(gw, one["d_weight"]) and torch.equal(gh, one["d_h"] + torch.ones_like(h))
    with pytest.raises(TypeError):
        residual_norm(h, y, out={})


def test_what_the_backward_needs_may_not_change(lp):
    from lm_head_linear_tcgen05_gb300.autograd import residual_norm
    h, y, w, _, _, _ = case(4, 64, BF, BF, False, "none", 3)
    w.requires_grad_()
    h_out, n = residual_norm(h, y, weight=w)
    h_out.add_(1)
    with pytest.raises(RuntimeError):
        n.sum().backward()


def test_refusals_of_the_binding(lp):
    h, y, w, wp, z, _ = case(4, 64, BF, BF, True, "channel", 3)
    f = lp.lp_residual_norm
    for kw, error in ((dict(weight=w.float(), gate=z), TypeError), (dict(weight=w[:32]), ValueError),
                      (dict(gate=torch.ones(4, 1, dtype=BF, device="cuda")), TypeError), (dict(gate=y[:, :32]), ValueError),
                      (dict(post_weight=wp), lp.LPError), (dict(eps=0.0), lp.LPError), (dict(eps=float("nan")), lp.LPError),
                      (dict(dropout=1.5), lp.LPError), (dict(dropout=-0.1), lp.LPError), (dict(row_start=-1), lp.LPError),
                      (dict(residual_scale=float("inf")), lp.LPError), (dict(norm_dtype=F32), TypeError),
                      (dict(norm=False, weight=w), lp.LPError), (dict(weight=w.cpu()), ValueError), (dict(eps="x"), TypeError),
                      (dict(row_start=1 << 63), TypeError), (dict(out=dict(norm=torch.empty_like(y)), norm=False), ValueError)):
        with pytest.raises(error):
            f(h, y, **kw)
    with pytest.raises(lp.LPError):
        f(h, dropout=0.5)
    with pytest.raises(lp.LPError):
        f(h[:, 4:60].as_strided((4, 56), (64, 1)), None)                    # rows off their 16-byte boundaries
    with pytest.raises(ValueError):
        f(h, y[:3])
    with pytest.raises(ValueError):
        f(h, y.t().contiguous().t())
    with pytest.raises(TypeError):
        f(h.half(), y)
    with pytest.raises(lp.LPError):
        lp.lp_residual_norm_backward(h, y, None, None)
    with pytest.raises(ValueError):
        lp.lp_residual_norm_backward(h, y, h, h, out=dict(d_gate=z))
    small = torch.empty(16, dtype=torch.uint8, device="cuda")
    lp.lp_residual_norm_backward(h, y, h, h, weight=w, workspace=small)          # a short batch needs none
    long = torch.zeros(300, 64, dtype=BF, device="cuda")
    with pytest.raises(lp.LPError):
        lp.lp_residual_norm_backward(long, long, long, long, weight=w, workspace=small)
    for kw in (dict(p=float("nan")), dict(p=2.0), dict(p=0.5, row_start=-2)):
        with pytest.raises(lp.LPError):
            lp.lp_dropout(h, seed=1, **kw)
    with pytest.raises(TypeError):
        lp.lp_dropout(h, 0.5, 1, rng=torch.zeros(2, dtype=torch.int32, device="cuda"))
    assert lp.lp_get_device_error() == 0


@pytest.mark.parametrize("limit", [1000, 20000])
@pytest.mark.parametrize("T,H", [(2000, 4096), (700, 8200), (20, 1032)])
def test_waits_that_run_out_are_recorded(lp, limit, T, H):
    """With a limit that few copies meet the call ends with LP_ERR_DEVICE_TIMEOUT, or in time; the next one, with the
    usual limit, is as if it had not been."""
    h, y, w, wp, z, gen = case(T, H, BF, BF, True, "channel", 7)
    o = dict(weight=w, post_norm=True, post_weight=wp, gate=z, dropout=0.1)
    dn, dh = rows(T, H, BF, gen), rows(T, H, BF, gen)
    both = lambda: (lp.lp_residual_norm(h, y, **o), lp.lp_residual_norm_backward(h, y, dn, dh, **o))  # noqa: E731
    want = both()
    assert lp.lp_get_device_error() == 0
    try:
        lp.lp_set_wait_limit(limit)
        both()
        assert lp.lp_get_device_error() in (0, 7)
    finally:
        lp.lp_set_wait_limit(0)
    got = both()
    assert lp.lp_get_device_error() == 0
    assert torch.equal(got[0][0], want[0][0]) and torch.equal(got[0][1], want[0][1])
    assert all(v is None or torch.equal(v, want[1][k]) for k, v in got[1].items())
