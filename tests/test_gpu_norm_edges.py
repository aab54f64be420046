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
