"""The bounds-checked build and the sorted positions of the embedding's gradient: a position whose key has no row
is not passed over in silence."""
import pytest

pytestmark = pytest.mark.gpu


def test_a_row_past_the_table_is_recorded():
    """The self-test asks for such a row as the summing kernels do, and records LP_ERR_BOUNDS only if that was
    noticed; the regular build refuses the row and records nothing."""
    import torch
    from lm_head_linear_tcgen05_gb300 import _build
    import lm_head_linear_tcgen05_gb300 as lp
    regular, debug = _build.build(), _build.build(debug_bounds=True)
    torch.cuda.set_device(0)
    try:
        lp.use_library(debug)
        lp.lp_selftest_bounds()
        assert lp.lp_get_device_error() == 10
    finally:
        lp.use_library(regular)
    lp.lp_selftest_bounds()
    assert lp.lp_get_device_error() == 0
