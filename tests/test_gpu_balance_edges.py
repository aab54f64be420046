"""lp_balance_loss where its inputs leave the ordinary range: gradients from upstream that are not finite, experts out of
reach under sigmoid scores, counts past 24 bits. Definition and bounds are block_ref.py's."""
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


def make(T, E, K, dtype, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    logits = torch.empty((T, E), dtype=dtype, device="cuda").normal_(0.0, 1.5, generator=gen)
    ids = torch.randint(0, E, (T, K), device="cuda", generator=gen, dtype=torch.int32)
    return logits, ids, (torch.rand(T, device="cuda", generator=gen) < 0.7).to(torch.uint8)


def offsets(*cu):
    return torch.tensor(cu, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("T", [24, 9000])               # one launch, several
@pytest.mark.parametrize("dtype,E,score,z", [(F32, 64, "softmax", 0.1), (BF, 64, "sigmoid", 0.0), (F32, 37, "softmax", 0.0)])
@pytest.mark.parametrize("up,coef", [(INF, 1.0), (-INF, 1.0), (NAN, 1.0), (3e38, 1e6)])
def test_what_is_not_kept_has_a_zero_gradient_whatever_is_upstream(lp, T, dtype, E, score, z, up, coef):
    logits, ids, mask = make(T, E, 4, dtype, T + E)
    o = dict(coef=coef, z_coef=z, score=score, mask=mask, upstream=torch.tensor([up], device="cuda"))
    for cu in (None, offsets(0, T // 3, T)):
        got = lp.lp_balance_loss(logits, ids, cu_seqlens=cu, **o)
        assert lp.lp_get_device_error() == 0
        assert bool((got["grad_logits"][mask == 0] == 0).all()) and bool(torch.isfinite(got["metrics"]).all())
        assert not bool(torch.isfinite(got["grad_logits"][mask != 0]).all())
    got = lp.lp_balance_loss(logits, ids, cu_seqlens=offsets(0, T // 2, T // 3, T), **o)
    assert lp.lp_get_device_error() == 12                 # gradients are zero, all of them
    assert bool((got["grad_logits"] == 0).all()) and bool(torch.isnan(got["metrics"]).all())


@pytest.mark.parametrize("by_sequence", [False, True])
def test_even_loads_past_24_bits_have_no_gradient(lp, by_sequence):
    """K N = 3 * 5592407 is odd and past 2^24, so no fp32 number; c E is the same number."""
    T = 5592407
    logits, _, _ = make(T, 3, 3, F32, 1)
    ids = torch.arange(3, device="cuda", dtype=torch.int32).repeat(T, 1)
    out = lp.lp_balance_loss(logits, ids, cu_seqlens=offsets(0, T) if by_sequence else None)
    assert lp.lp_get_device_error() == 0
    assert out["expert_counts"].tolist() == [T] * 3 and float(out["grad_logits"].abs().max()) == 0.0


@pytest.mark.parametrize("by_sequence", [False, True])
@pytest.mark.parametrize("T,K,E", [(1000003, 63, 3), (1000003, 64, 2)])
def test_counts_past_24_bits(lp, T, K, E, by_sequence):
    """Experts named about evenly, each more than 2^24 times: f - 1 is some 1e-4, of which a count rounded to fp32 would
    leave three digits."""
    logits, ids, _ = make(T, E, K, F32, 2)
    cu = offsets(0, T) if by_sequence else None
    out = lp.lp_balance_loss(logits, ids, coef=0.7, cu_seqlens=cu)
    metrics, experts, counts, grad, m_tol, g_tol = ref.balance(logits, ids, 0.7, cu=cu)
    assert int(experts.min()) > 1 << 24 and torch.equal(out["expert_counts"], experts) and torch.equal(out["counts"], counts)
    assert bool(((out["metrics"].double() - metrics).abs() <= m_tol + ref.U * metrics.abs()).all())
    assert bool(((out["grad_logits"].double() - grad).abs() <= g_tol + ref.U * (grad.abs() + g_tol) + 1e-37).all())
    assert lp.lp_get_device_error() == 0


@pytest.mark.parametrize("T", [24, 9000])
@pytest.mark.parametrize("dtype,E", [(F32, 64), (BF, 64), (F32, 37), (BF, 37), (F32, 260)])
def test_a_sigmoid_score_of_minus_infinity_is_zero(lp, T, dtype, E):
    """1 / (1 + e^inf) = 0: such an expert has no probability and no gradient, however small the others' scores are."""
    logits, ids, _ = make(T, E, 4, dtype, T + E)
    logits[:, 3:7] = -INF
    logits[1, :] -= 44.0                                  # scores of about e^-44: their sum is above what is rescaled
    logits[2, :] -= 80.0                                  # below it
    logits[3, :] = -INF
    out = lp.lp_balance_loss(logits, ids, coef=0.5, score="sigmoid")
    assert lp.lp_get_device_error() == 0
    gone = logits == -INF
    assert bool((out["grad_logits"][gone] == 0).all())
    metrics, _, _, grad, m_tol, g_tol = ref.balance(logits, ids, 0.5, 0.0, "sigmoid")
    got = out["grad_logits"]
    assert bool(((got.double() - grad).abs() <= g_tol + ref.HALF_STEP[dtype] * (grad.abs() + g_tol) + 1e-37).all())
    assert bool(((out["metrics"].double() - metrics).abs() <= m_tol + ref.U * metrics.abs() + 1e-37).all())
