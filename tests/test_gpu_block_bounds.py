"""The operators between the embedding and the losses in the bounds-checked build, which has to find nothing and give the
regular build's bits; waits that run out (there the norms' waits poll, so that a limit of a microsecond is kept; in the
regular build the hardware suspends a waiting thread for longer than a row takes to arrive); and canary words around a
workspace of exactly the size asked for and around the outputs that are vectors."""
import itertools

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


def both_builds(libs, run):
    """What run() returns, from either build; the bounds-checked one must find nothing."""
    lp, regular, debug = libs
    lp.use_library(regular)
    want = run()
    assert lp.lp_get_device_error() == 0
    lp.use_library(debug)
    assert lp.lp_debug_bounds_build()
    got = run()
    assert lp.lp_get_device_error() == 0
    lp.use_library(regular)
    assert same(got, want)


# both sides of the widths and batches where another kernel takes over
NORMS = [(1, 8), (256, 64), (257, 64), (70, 72), (64, 256), (65, 256), (24, 1032), (25, 1032), (400, 4104), (24, 8192), (2, 8200),
         (333, 8200), (160, 16384), (5001, 136)]


@pytest.mark.parametrize("T,H", NORMS)
@pytest.mark.parametrize("stream,branch,gate,post,p", [(BF, BF, "channel", True, 0.1), (F32, BF, "token", False, 0.1),
                                                       (F32, F32, "full", True, 0.0), (BF, F32, "none", False, 0.0)])
def test_norms_pass_the_bounds_checks(libs, T, H, stream, branch, gate, post, p):
    lp = libs[0]
    gen = torch.Generator(device="cuda").manual_seed(T + H)
    rows = lambda dt: torch.empty((T, H + 24), dtype=dt, device="cuda").normal_(generator=gen)[:, :H]    # noqa: E731
    vec = lambda: torch.empty(H, dtype=branch, device="cuda").normal_(generator=gen)                     # noqa: E731
    h, y, dn, dh = rows(stream), rows(branch), rows(branch), rows(stream)
    z = {"none": lambda: None, "channel": vec, "token": lambda: torch.rand((T, 1), device="cuda", generator=gen),
         "full": lambda: rows(branch)}[gate]()
    o = dict(weight=vec(), post_norm=post, post_weight=vec() if post else None, gate=z, dropout=p, seed=5)

    def run():
        out = list(lp.lp_residual_norm(h, y, **o)) + list(lp.lp_residual_norm(h, weight=o["weight"], norm_dtype=branch))
        out += lp.lp_residual_norm_backward(h, y, dn, dh, **o).values()
        out += lp.lp_residual_norm_backward(h, y, None, dh, **o).values()
        out += lp.lp_residual_norm_backward(h, None, dn, None, weight=o["weight"]).values()
        return out + [lp.lp_dropout(h, 0.3, 7), lp.lp_dropout(dn.contiguous(), 0.3, 7, row_start=11)]
    both_builds(libs, run)


BALANCE = [(1, 1, 1, None), (37, 64, 8, None), (300, 60, 3, [100, 0, 199, 1]), (4096, 64, 8, None), (4097, 64, 8, None),
           (30, 1024, 16, [1] * 30), (6000, 37, 5, [3, 0, 5, 1, 1] * 600), (70001, 128, 8, None), (9000, 256, 4, [4000, 0, 4999, 1]),
           (9000, 1024, 2, [9000])]


@pytest.mark.parametrize("T,E,K,lengths", BALANCE)
@pytest.mark.parametrize("dtype,score,pad", [(F32, "softmax", 0), (BF, "sigmoid", 8), (F32, "sigmoid", 1)])
def test_balance_passes_the_bounds_checks(libs, T, E, K, lengths, dtype, score, pad):
    lp = libs[0]
    gen = torch.Generator(device="cuda").manual_seed(T + E)
    logits = torch.empty((T, E + pad), dtype=dtype, device="cuda").normal_(generator=gen)[:, :E]
    ids = torch.randint(-1, E, (T, K), device="cuda", generator=gen, dtype=torch.int32)
    mask = (torch.rand(T, device="cuda", generator=gen) < 0.8).to(torch.uint8)
    cu = None if lengths is None else torch.tensor([0, *itertools.accumulate(lengths)], dtype=torch.int32, device="cuda")

    def run():
        r = lp.lp_balance_loss(logits, ids, score=score, mask=mask, cu_seqlens=cu)
        return [r[k] for k in ("metrics", "expert_counts", "counts", "grad_logits")]
    both_builds(libs, run)


class Guarded:
    """n bytes between words that nothing writes."""

    def __init__(self, n, dtype=torch.uint8):
        self.bytes = torch.full((n + 2048,), 0xA5, dtype=torch.uint8, device="cuda")
        self.inner = self.bytes[1024:1024 + n].view(dtype)
        self.n = n

    def intact(self):
        return bool((self.bytes[:1024] == 0xA5).all()) and bool((self.bytes[1024 + self.n:] == 0xA5).all())


@pytest.mark.parametrize("T,H", NORMS)
@pytest.mark.parametrize("dw", [F32, BF])
def test_the_norms_gradient_keeps_to_its_workspace_and_vectors(libs, T, H, dw):
    lp = libs[0]
    gen = torch.Generator(device="cuda").manual_seed(T + H)
    rows = lambda: torch.empty((T, H), dtype=BF, device="cuda").normal_(generator=gen)                   # noqa: E731
    vec = lambda: torch.empty(H, dtype=BF, device="cuda").normal_(generator=gen)                         # noqa: E731
    h, y, dn, dh, w, wp = rows(), rows(), rows(), rows(), vec(), vec()
    for gate in (vec(), torch.rand((T, 1), device="cuda", generator=gen)):
        ws = Guarded(lp.lp_norm_workspace_size(T, H))
        names = ["d_weight", "d_post_weight"] + (["d_gate"] if gate.dim() == 1 else [])
        vectors = {k: Guarded(H * dw.itemsize, dw) for k in names}
        out = {k: v.inner for k, v in vectors.items()}
        if gate.dim() == 2:
            vectors["d_gate"] = Guarded(4 * T, F32)
            out["d_gate"] = vectors["d_gate"].inner.view(T, 1)
        o = dict(weight=w, post_norm=True, post_weight=wp, gate=gate, dw_dtype=dw)
        want = lp.lp_residual_norm_backward(h, y, dn, dh, **o)
        got = lp.lp_residual_norm_backward(h, y, dn, dh, out=out, workspace=ws.inner, **o)
        assert lp.lp_get_device_error() == 0
        assert ws.intact() and all(v.intact() for v in vectors.values())
        assert all(torch.equal(got[k], want[k]) for k in want)


@pytest.mark.parametrize("T,E,K,lengths", BALANCE)
def test_the_balance_loss_keeps_to_its_workspace_and_vectors(libs, T, E, K, lengths):
    lp = libs[0]
    gen = torch.Generator(device="cuda").manual_seed(T + E)
    logits = torch.empty((T, E), device="cuda").normal_(generator=gen)
    ids = torch.randint(-1, E, (T, K), device="cuda", generator=gen, dtype=torch.int32)
    cu = None if lengths is None else torch.tensor([0, *itertools.accumulate(lengths)], dtype=torch.int32, device="cuda")
    S = 0 if lengths is None else len(lengths)
    ws = Guarded(lp.lp_balance_workspace_size(T, E, K, S))
    want = lp.lp_balance_loss(logits, ids, coef=0.5, cu_seqlens=cu)
    metrics, experts, counts, grad = Guarded(16, F32), Guarded(8 * E, torch.int64), Guarded(16, torch.int64), Guarded(4 * T * E, F32)
    st = lp.lib().lp_balance_loss(
        T, E, K, lp._BALANCE_INPUTS.pack(logits.data_ptr(), ids.data_ptr(), 0, 0 if cu is None else cu.data_ptr(), 0, E, S),
        lp._BALANCE_OPTIONS.pack(0.5, 0.0, 0, lp.LP_DTYPE_F32, lp.LP_DTYPE_F32),
        lp._BALANCE_OUTPUTS.pack(metrics.inner.data_ptr(), experts.inner.data_ptr(), counts.inner.data_ptr(),
                                 grad.inner.data_ptr(), E),
        ws.inner.data_ptr(), ws.n, torch.cuda.current_stream().cuda_stream)
    assert st == 0 and lp.lp_get_device_error() == 0
    assert all(b.intact() for b in (ws, metrics, experts, counts, grad))
    assert torch.equal(metrics.inner, want["metrics"]) and torch.equal(experts.inner, want["expert_counts"])
    assert torch.equal(counts.inner, want["counts"]) and torch.equal(grad.inner.view(T, E), want["grad_logits"])
