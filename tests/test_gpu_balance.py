"""lp_balance_loss on the GPU against its 64-bit definition (block_ref.py), under bounds that count the roundings of
exponents, powers, sums and the gradient's type."""
import itertools
import random

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
import block_ref as ref  # noqa: E402

BF, F32 = torch.bfloat16, torch.float32
NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module")
def lp():
    from lm_head_linear_tcgen05_gb300 import _build
    _build.build()
    import lm_head_linear_tcgen05_gb300 as mod
    assert mod.lp_device_supported()
    torch.cuda.set_device(0)
    return mod


def make(T, E, K, dtype, seed, lengths=None, masked=0.3, std=1.5, pad=0, shift=0):
    """logits in a wider buffer, ids, mask, offsets; NaN, infinities and wrong ids where the mask drops a token."""
    gen = torch.Generator(device="cuda").manual_seed(seed)
    buffer = torch.full((T * (E + pad) + shift,), NAN, dtype=dtype, device="cuda")
    logits = buffer[shift:].view(T, E + pad)[:, :E]
    logits.normal_(0.0, std, generator=gen)
    ids = torch.rand((T, E), device="cuda", generator=gen).argsort(1)[:, :K].to(torch.int32)
    if K > E:
        ids = torch.randint(0, E, (T, K), device="cuda", generator=gen, dtype=torch.int32)
    ids = torch.where(torch.rand((T, K), device="cuda", generator=gen) < 0.1, -1, ids).to(torch.int32).contiguous()
    mask = None
    if masked:
        mask = (torch.rand(T, device="cuda", generator=gen) >= masked).to(torch.uint8)
        drop = mask == 0
        junk = torch.tensor([NAN, INF, -INF], device="cuda")
        logits[drop] = junk[torch.randint(0, 3, (int(drop.sum()), E), device="cuda", generator=gen)].to(dtype)
        ids[drop] = 1 << 20
    cu = None
    if lengths is not None:
        cu = torch.tensor([0] + list(itertools.accumulate(lengths)), dtype=torch.int32, device="cuda")
        assert int(cu[-1]) == T
    return logits, ids, mask, cu


def check(lp, logits, ids, mask, cu, coef=0.7, z=0.0, score="softmax", up=None, **kw):
    out = lp.lp_balance_loss(logits, ids, coef=coef, z_coef=z, score=score, mask=mask, cu_seqlens=cu,
                             upstream=None if up is None else torch.tensor([up], device="cuda"), **kw)
    metrics, experts, counts, grad, m_tol, g_tol = ref.balance(logits, ids, coef, z, score, mask, cu)
    assert torch.equal(out["expert_counts"], experts) and torch.equal(out["counts"], counts)
    metrics = torch.where(metrics.float().isinf(), metrics.float(), metrics)       # past the largest fp32 value
    over = (out["metrics"].double() - metrics).abs() / (m_tol + ref.U * metrics.abs() + 1e-37)
    over[out["metrics"] == metrics] = 0.0
    assert float(over.max()) <= 1.0, ("metrics", over.tolist())
    up = 1.0 if up is None else up
    grad, g_tol = up * grad, abs(up) * g_tol
    got = out["grad_logits"]
    over = (got.double() - grad).abs() / (g_tol + ref.HALF_STEP[got.dtype] * (grad.abs() + g_tol) + 1e-37)
    worst = float(over.max()) if over.numel() else 0.0
    assert worst <= 1.0, ("gradient", worst)
    assert lp.lp_get_device_error() == 0
    return out


EXPERTS = [1, 2, 3, 7, 8, 16, 17, 32, 33, 60, 64, 65, 72, 128, 129, 160, 200, 256, 264, 371, 512, 513, 520, 1000, 1024]


@pytest.mark.parametrize("E", EXPERTS)
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("dtype", [F32, BF])
def test_every_width(lp, E, score, dtype):
    rnd = random.Random(E)
    for T, K, lengths, pad, shift in ((1, 1, None, 0, 0), (37, min(E, 8), None, 0, 0), (50, min(E, 3), [20, 0, 29, 1, 0], 8, 0),
                                      (45, min(E, 2), [45], 1, 1), (24, min(E, 4), [1] * 24, 0, 0)):
        logits, ids, mask, cu = make(T, E, K, dtype, E + T, lengths, rnd.choice((0.0, 0.3)), pad=pad, shift=shift)
        check(lp, logits, ids, mask, cu, z=0.01 if score == "softmax" else 0.0, score=score, up=rnd.choice((None, 3.0, -0.5)))


LENGTHS = {
    "even": [4096] * 4, "ragged": [9000, 0, 1, 3000, 5, 0, 0, 4000, 378], "short": [3, 0, 5, 1, 2] * 1490, "mixed": [8000] + [2, 0, 7] * 931,
}


@pytest.mark.parametrize("lengths", list(LENGTHS))
@pytest.mark.parametrize("E,K,dtype,score", [(64, 8, F32, "softmax"), (256, 4, BF, "sigmoid"), (37, 5, F32, "sigmoid"), (128, 1, BF, "softmax")])
def test_long_batches_by_sequence(lp, lengths, E, K, dtype, score):
    lengths = LENGTHS[lengths]
    logits, ids, mask, cu = make(sum(lengths), E, K, dtype, 3, lengths)
    a = check(lp, logits, ids, mask, cu, score=score, z=0.02 if score == "softmax" else 0.0)
    b = lp.lp_balance_loss(logits, ids, coef=0.7, score=score, mask=mask, cu_seqlens=cu, z_coef=0.02 if score == "softmax" else 0.0)
    for k in ("metrics", "expert_counts", "counts", "grad_logits"):
        assert torch.equal(a[k], b[k]), k


@pytest.mark.parametrize("T,E,K,dtype,score", [(5000, 64, 8, F32, "softmax"), (70001, 128, 8, F32, "softmax"), (40000, 9, 2, BF, "softmax"),
                                               (33000, 200, 64, F32, "sigmoid"), (3001, 1024, 16, BF, "sigmoid"), (150000, 2, 1, F32, "softmax")])
def test_long_batches(lp, T, E, K, dtype, score):
    logits, ids, mask, _ = make(T, E, K, dtype, T, masked=0.1)
    check(lp, logits, ids, mask, None, coef=0.01, score=score, z=0.001 if score == "softmax" else 0.0)
    check(lp, logits, ids, mask, None, coef=0.0, score=score, z=1.0 if score == "softmax" else 0.0)


@pytest.mark.parametrize("T", [20, 6000])
@pytest.mark.parametrize("by_sequence", [False, True])
def test_nothing_kept(lp, T, by_sequence):
    logits, ids, _, cu = make(T, 64, 2, F32, 1, [T // 2, T - T // 2] if by_sequence else None, masked=0)
    logits.fill_(NAN)
    out = check(lp, logits, ids, torch.zeros(T, dtype=torch.bool, device="cuda"), cu)
    assert float(out["metrics"].abs().max()) == 0.0 and float(out["grad_logits"].abs().max()) == 0.0


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("T", [16, 9000])
def test_extreme_logits(lp, score, T):
    """-inf for experts out of reach, a token without any, the type's lowest value, logits whose scores all but vanish."""
    logits, ids, _, _ = make(T, 64, 4, F32, 2, masked=0)
    logits[:, 5:9] = -INF
    logits[1] = -INF
    logits[2] = -3.4028234663852886e38
    logits[3] = logits[3] - 120.0
    logits[4] = logits[4] * 0.1 - 60.0
    logits[5] = logits[5] + 90.0
    logits[6, :] = -200.0
    logits[6, 11] = -195.0
    ids[1] = -1
    out = check(lp, logits, ids, None, None, score=score)
    assert float(out["grad_logits"][1].abs().max()) == 0.0
    # the square of the lowest value's log-sum-exp is past fp32, and 0 times it does not enter the loss
    assert torch.isfinite(out["metrics"]).tolist() == [True, True, score == "sigmoid", True]
    if score == "softmax":
        assert float(out["grad_logits"][logits == -INF].abs().max()) == 0.0


@pytest.mark.parametrize("T", [30, 20000])
@pytest.mark.parametrize("bad", [NAN, INF])
def test_a_row_that_is_not_finite_leaves_the_others(lp, T, bad):
    logits, ids, mask, _ = make(T, 128, 8, F32, 4, masked=0)
    want = lp.lp_balance_loss(logits, ids, coef=0.5)["grad_logits"].clone()
    logits[7, 3] = bad
    out = lp.lp_balance_loss(logits, ids, coef=0.5)
    good = torch.arange(T, device="cuda") != 7
    assert torch.equal(out["grad_logits"][good], want[good]) and bool(torch.isnan(out["metrics"][0]))
    assert bool(torch.isnan(out["grad_logits"][7]).any())


@pytest.mark.parametrize("T", [24, 20000])
def test_evenly_used_experts(lp, T):
    """With every expert named equally often the gradient is exactly zero, whatever the logits."""
    logits, _, _, _ = make(T, 8, 2, F32, 2, masked=0)
    ids = torch.arange(2 * T, device="cuda", dtype=torch.int32).remainder(8).view(T, 2)
    out = lp.lp_balance_loss(logits, ids)
    assert float(out["grad_logits"].abs().max()) == 0.0 and abs(float(out["loss"]) - 1.0) < 64 * ref.U
    assert out["metrics"].tolist()[3] == 1.0


@pytest.mark.parametrize("T", [40, 12000])
def test_outputs_that_are_asked_for(lp, T):
    logits, ids, mask, cu = make(T, 32, 4, F32, 9, [T // 3, T - T // 3], pad=8)
    o = dict(coef=0.3, mask=mask, cu_seqlens=cu)
    all_of = lp.lp_balance_loss(logits, ids, **o)
    only = lp.lp_balance_loss(logits, ids, grads=False, **o)
    assert torch.equal(only["metrics"], all_of["metrics"]) and only["grad_logits"] is None
    only = lp.lp_balance_loss(logits, ids, metrics=False, **o)
    assert torch.equal(only["grad_logits"], all_of["grad_logits"]) and only["metrics"] is None
    half = lp.lp_balance_loss(logits, ids, grad_dtype=BF, **o)["grad_logits"]
    assert torch.equal(half, all_of["grad_logits"].to(BF))
    wide = torch.full((T + 2, 40), 7.0, device="cuda")
    # off its 16-byte boundaries, so element by element: sums in another order
    check(lp, logits, ids, mask, cu, coef=0.3, out=wide[1:-1, 3:35])
    assert bool((wide[0] == 7).all() and (wide[-1] == 7).all() and (wide[:, :3] == 7).all() and (wide[:, 35:] == 7).all())
    buffer = logits.clone()
    got = lp.lp_balance_loss(buffer, ids, out=buffer, **o)
    assert got["grad_logits"] is buffer and torch.equal(buffer, all_of["grad_logits"])
    assert torch.equal(got["loss"], all_of["loss"]) and float(all_of["loss"]) == float(all_of["metrics"][0])


def test_empty_batch(lp):
    out = lp.lp_balance_loss(torch.empty(0, 16, device="cuda"), torch.empty(0, 2, dtype=torch.int32, device="cuda"))
    assert out["metrics"].tolist() == [0.0] * 4 and out["counts"].tolist() == [0, 0] and out["grad_logits"].shape == (0, 16)
    assert int(out["expert_counts"].abs().sum()) == 0


@pytest.mark.parametrize("T", [64, 9000])
@pytest.mark.parametrize("by_sequence", [False, True])
def test_ids_out_of_range_are_recorded_and_not_counted(lp, T, by_sequence):
    logits, ids, _, cu = make(T, 16, 2, F32, 3, [T // 2, T - T // 2] if by_sequence else None, masked=0)
    want = lp.lp_balance_loss(logits, torch.where(ids == 3, -1, ids).to(torch.int32), cu_seqlens=cu)
    for wrong in (16, -2, 1 << 30, -(1 << 31)):
        got = lp.lp_balance_loss(logits, torch.where(ids == 3, wrong, ids).to(torch.int32), cu_seqlens=cu)
        assert lp.lp_get_device_error() == 13
        for k in ("metrics", "expert_counts", "counts", "grad_logits"):
            assert torch.equal(got[k], want[k]), (wrong, k)


@pytest.mark.parametrize("T", [64, 9000])
@pytest.mark.parametrize("cu", [[0, 10, 5, -1], [1, 20, -1], [0, 20, -2], [0, -7, -1], [0, 1 << 30, -1]])
def test_offsets_out_of_order(lp, T, cu):
    logits, ids, _, _ = make(T, 16, 2, F32, 3, masked=0)
    cu = torch.tensor([T if c == -1 else T - 1 if c == -2 else c for c in cu], dtype=torch.int32, device="cuda")
    out = lp.lp_balance_loss(logits, ids, cu_seqlens=cu)
    assert lp.lp_get_device_error() == 12
    assert bool(torch.isnan(out["metrics"]).all()) and float(out["grad_logits"].abs().max()) == 0.0


@pytest.mark.parametrize("T", [64, 9000])
def test_a_captured_call_reads_its_inputs_again(lp, T):
    logits, ids, mask, cu = make(T, 64, 4, F32, 3, [T // 4, T - T // 4])
    ids[mask == 0] = 0
    up = torch.ones(1, device="cuda")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    o = dict(coef=0.5, z_coef=0.1, mask=mask, cu_seqlens=cu, upstream=up)
    with torch.cuda.stream(s):
        lp.lp_balance_loss(logits, ids, **o)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            got = lp.lp_balance_loss(logits, ids, **o)
    torch.cuda.current_stream().wait_stream(s)
    for step in (1, 2):
        logits.copy_(torch.randn_like(logits))
        up.fill_(float(step))
        ids.copy_(ids.roll(1, 0))
        graph.replay()
        want = lp.lp_balance_loss(logits, ids, **o)
        for k in ("metrics", "expert_counts", "counts", "grad_logits"):
            assert torch.equal(got[k], want[k]), k


def test_two_streams_at_once(lp):
    cases = [make(20000, 128, 8, F32, 1), make(30000, 64, 4, BF, 2, [10000, 20000])]
    run = lambda c: lp.lp_balance_loss(c[0], c[1], mask=c[2], cu_seqlens=c[3])  # noqa: E731
    want = [run(c) for c in cases]
    streams = [torch.cuda.Stream() for _ in cases]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(5):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i].append(run(cases[i]))
    torch.cuda.synchronize()
    for i in range(2):
        for r in got[i]:
            for k in ("metrics", "expert_counts", "counts", "grad_logits"):
                assert torch.equal(r[k], want[i][k]), k


@pytest.mark.parametrize("T,lengths", [(50, None), (9000, [4000, 5000])])
def test_autograd(lp, T, lengths):
    from lm_head_linear_tcgen05_gb300.autograd import balance_loss
    logits, ids, mask, cu = make(T, 64, 4, BF, 5, lengths)
    o = dict(coef=0.2, z_coef=0.03, mask=mask, cu_seqlens=cu)
    logits.requires_grad_()
    loss, metrics, experts, counts = balance_loss(logits, ids, **o)
    (g,) = torch.autograd.grad(3.0 * loss, (logits,))
    want = lp.lp_balance_loss(logits.detach(), ids, upstream=torch.tensor([3.0], device="cuda"), **o)
    assert g.dtype is BF and torch.equal(g, want["grad_logits"]) and torch.equal(metrics, want["metrics"])
    assert torch.equal(experts, want["expert_counts"]) and torch.equal(counts, want["counts"]) and float(loss.detach()) == float(metrics[0])
    for name in ("upstream", "grads", "metrics", "out", "grad_dtype"):
        with pytest.raises(TypeError):
            balance_loss(logits, ids, **{name: None})


def test_refusals_of_the_binding(lp):
    logits, ids, _, cu = make(20, 16, 2, F32, 1, [20], masked=0)
    f = lp.lp_balance_loss
    for a, kw, error in (((logits.double(), ids), {}, TypeError), ((logits.cpu(), ids), {}, TypeError), ((logits, ids.long()), {}, TypeError),
                         ((logits, ids[:10]), {}, ValueError), ((logits, ids.t().contiguous().t()), {}, ValueError),
                         ((logits.t(), ids), {}, ValueError), ((logits, ids), dict(score="other"), ValueError),
                         ((logits, ids), dict(coef=NAN), lp.LPError), ((logits, ids), dict(score="sigmoid", z_coef=0.1), lp.LPError),
                         ((logits, ids), dict(mask=torch.ones(19, dtype=torch.bool, device="cuda")), ValueError),
                         ((logits, ids), dict(cu_seqlens=cu.long()), TypeError), ((logits, ids), dict(cu_seqlens=cu[:1]), lp.LPError),
                         ((logits, ids), dict(out=logits, grads=False), ValueError), ((logits, ids), dict(grad_dtype=torch.half), TypeError),
                         ((logits, ids), dict(grads=False, metrics=False), lp.LPError), ((logits, ids), dict(coef="x"), TypeError),
                         ((logits, ids), dict(upstream=torch.ones(2, device="cuda")), TypeError),
                         ((torch.zeros(20, 1025, device="cuda"), ids), {}, lp.LPError),
                         ((logits, torch.zeros(20, 65, dtype=torch.int32, device="cuda")), {}, lp.LPError)):
        with pytest.raises(error):
            f(*a, **kw)
    big, ids, _, _ = make(9000, 64, 2, F32, 1, masked=0)
    with pytest.raises(lp.LPError):
        f(big, ids, workspace=torch.empty(64, dtype=torch.uint8, device="cuda"))
    assert lp.lp_get_device_error() == 0
