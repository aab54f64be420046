"""The operators between the embedding and the losses in the bounds-checked build: waits that run out (there the norms'
waits poll, so that a limit of a microsecond is kept; in the regular build the hardware suspends a waiting thread for
longer than a row takes to arrive)."""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def libs():
    from lm_head_linear_tcgen05_gb300 import _build
    regular, debug = _build.build(), _build.build(debug_bounds=True)
    import lm_head_linear_tcgen05_gb300 as mod
    assert mod.lp_device_supported()
    torch.cuda.set_device(0)
    yield mod, regular, debug
    mod.use_library(regular)          # later test modules run on the regular build


def same(a, b):
    return all((x is None and y is None) or torch.equal(x, y) for x, y in zip(a, b, strict=True))


# A row of the first three is 48 to 196 KB a CTA, of inputs past the L2: 152 or 304 of them asked for at once take some
# 4 us at the rate of the memory and 1.3 us at the most an SM takes in, and the CTA has nothing else to do meanwhile. The
# fourth has up to three rows in flight and is bound by memory. 16384 columns of a gradient belong to two CTAs.
@pytest.mark.parametrize("T,H,dtype,gate", [(2000, 4096, F32, True), (1500, 8192, F32, True), (1000, 16384, F32, True),
                                            (4000, 8192, BF, False)])
def test_waits_that_run_out_end_the_call(libs, T, H, dtype, gate):
    lp, regular, debug = libs
    gen = torch.Generator(device="cuda").manual_seed(H)
    rows = lambda: torch.empty((T, H), dtype=dtype, device="cuda").normal_(generator=gen)  # noqa: E731
    h, y, dn, dh, z = rows(), rows(), rows(), rows(), rows() if gate else None
    w = torch.empty(H, dtype=dtype, device="cuda").normal_(generator=gen)
    forward = lambda: lp.lp_residual_norm(h, y, weight=w, gate=z)                                        # noqa: E731
    backward = lambda: tuple(lp.lp_residual_norm_backward(h, y, dn, dh, weight=w, gate=z).values())      # noqa: E731
    lp.use_library(regular)
    want = forward(), backward()
    assert lp.lp_get_device_error() == 0
    lp.use_library(debug)
    try:
        lp.lp_set_wait_limit(1000)
        for call in (forward, backward):
            seen = []
            for _ in range(6):
                call()
                seen.append(lp.lp_get_device_error())
            assert set(seen) <= {0, 7} and 7 in seen          # LP_ERR_DEVICE_TIMEOUT
    finally:
        lp.lp_set_wait_limit(0)
    got = forward(), backward()
    assert lp.lp_get_device_error() == 0
    lp.use_library(regular)
    assert same(got[0], want[0]) and same(got[1], want[1])
