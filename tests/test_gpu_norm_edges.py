"""Refusals of lp_residual_norm and lp_dropout that could have passed for another call, and batches of more than 2^31
elements of the norms, dropout and the balance loss."""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def lp():
    from lm_head_linear_tcgen05_gb300 import _build
    _build.build()
    import lm_head_linear_tcgen05_gb300 as mod
    assert mod.lp_device_supported()
    torch.cuda.set_device(0)
    return mod


@pytest.mark.parametrize("start", [-1, 1 << 63, (1 << 64) + 7, -(1 << 64) + 7])
def test_a_first_row_past_63_bits_is_refused(lp, start):
    x = torch.ones(4, 64, device="cuda")
    for call in (lambda: lp.lp_dropout(x, 0.5, 1, row_start=start), lambda: lp.lp_residual_norm(x, x, dropout=0.5, row_start=start)):
        with pytest.raises((TypeError, lp.LPError)):
            call()


def test_an_output_of_another_name_is_refused(lp):
    h = torch.ones(4, 64, device="cuda")
    for name in ("d_h", "hout", "y"):
        with pytest.raises(ValueError):
            lp.lp_residual_norm(h, h, out={name: torch.empty_like(h)})


T_BIG, H_BIG = 600001, 4096                                # 2.46e9 elements, 4.9 GB in bf16


def big_rows(seed, last):
    """A matrix of zeros but for its first and last `last` rows."""
    gen = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.zeros((T_BIG, H_BIG), dtype=BF, device="cuda")
    for part in (x[:last], x[-last:]):
        part.normal_(generator=gen)
    return x


def test_norms_of_more_than_2_31_elements(lp):
    """The last rows are those of a call on them alone; the sums over tokens are of the rows that are not zero."""
    n, ones = 200, torch.ones(H_BIG, dtype=BF, device="cuda")
    h, y, dn, dh = (big_rows(s, n) for s in range(4))
    o = dict(weight=ones, post_norm=True, post_weight=ones, dropout=0.25, seed=9)
    end = [x[-n:].clone() for x in (h, y, dn, dh)]
    want = lp.lp_residual_norm(end[0], end[1], row_start=T_BIG - n, **o)
    got = lp.lp_residual_norm(h, y, **o)
    for a, b in zip(got, want):
        assert torch.equal(a[-n:], b) and not bool(a[n:-n:997].any())
    u = got[0]
    want = lp.lp_residual_norm_backward(u[-n:].clone(), end[1], end[2], end[3], row_start=T_BIG - n, **o)
    start = lp.lp_residual_norm_backward(u[:n].clone(), *(x[:n].clone() for x in (y, dn, dh)), **o)
    got = lp.lp_residual_norm_backward(u, y, dn, dh, **o)
    for k in ("d_h", "d_y"):
        assert torch.equal(got[k][-n:], want[k]) and torch.equal(got[k][:n], start[k])
    # 400 terms of d_weight in another order and grouping: each sum has at most 400 roundings of at most the sum of
    # their absolute values, which is below 400 max |dn| max |norm| = 400 * 6 * 6; rms is at most that over sqrt(400)
    both = want["d_weight"].double() + start["d_weight"].double()
    assert float((got["d_weight"].double() - both).abs().max()) <= 3 * 400 * 2.0 ** -24 * 400 * 36
    assert lp.lp_get_device_error() == 0


@pytest.mark.parametrize("pad", [0, 8])
def test_dropout_of_more_than_2_31_elements(lp, pad):
    n = 200
    x = torch.ones((T_BIG, H_BIG + pad), dtype=BF, device="cuda")[:, :H_BIG]
    got = lp.lp_dropout(x, 0.25, 9, offset=3)
    for at in (0, T_BIG // 2, (1 << 31) // H_BIG - 100, T_BIG - n):
        assert torch.equal(got[at:at + n], lp.lp_dropout(x[at:at + n], 0.25, 9, offset=3, row_start=at))
    assert lp.lp_get_device_error() == 0


@pytest.mark.parametrize("by_sequence", [False, True])
def test_balance_of_more_than_2_31_logits(lp, by_sequence):
    """The same logits in the same sequence have the same gradient, wherever they are; an expert is named by T / E tokens."""
    T, E, n = 2200000, 1024, 64                             # 2.25e9 logits, 9 GB
    logits = torch.zeros((T, E), device="cuda")
    logits[:n].normal_(generator=torch.Generator(device="cuda").manual_seed(1))
    logits[-n:] = logits[:n]
    ids = (torch.arange(T, device="cuda", dtype=torch.int32) % 1000).view(T, 1)
    cu = torch.tensor([0, T], dtype=torch.int32, device="cuda") if by_sequence else None
    out = lp.lp_balance_loss(logits, ids, cu_seqlens=cu)
    g = out["grad_logits"]
    assert torch.equal(g[-n:], g[:n]) and bool(g[:n].any(1).all())
    # a row of equal logits has p = 1 / E and sum f p = 1: its gradient is w p (f - 1), of which f - 1 = c E / T - 1 is
    # rounded three times, the mean over 1024 experts 10 times in each of p, f - 1 and their products' sum
    f = torch.bincount(ids.view(-1).long(), minlength=E).double() * E / T - 1
    want = f / E / T
    tol = 2.0 ** -24 * (4 * f.abs() + 64 * f.abs().mean()) / E / T
    for row in (n, T // 2, (1 << 31) // E + 1, T - n - 1):
        assert bool(((g[row].double() - want).abs() <= tol + 2.0 ** -24 * want.abs()).all())
    assert out["counts"].tolist() == [T, int(by_sequence)] and int(out["expert_counts"].sum()) == T
    assert lp.lp_get_device_error() == 0
