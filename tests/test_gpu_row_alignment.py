"""Rows that start on 16-byte boundaries but not on 32-byte ones, and gradients in other orders: the bits are those of
the aligned, contiguous call."""
import numpy as np
import pytest

from lp_util import dev_i32

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def lp():
    from lm_head_linear_tcgen05_gb300 import _build
    _build.build()
    import lm_head_linear_tcgen05_gb300 as mod
    import torch
    assert mod.lp_device_supported()
    torch.cuda.set_device(0)
    return mod


def _normal(shape, dtype, seed):
    import torch
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return torch.empty(shape, dtype=dtype, device="cuda").normal_(generator=g)


def _off32(rows, width, dtype, ld=None, fill=5.0):
    """A [rows, width] view of row stride ld that starts 16 bytes past a 32-byte boundary, and the buffer it lies in."""
    import torch
    ld = width if ld is None else ld
    skip = 4 if dtype == torch.float32 else 8
    buf = torch.full((skip + rows * ld + 64,), fill, dtype=dtype, device="cuda")
    view = buf[skip:skip + rows * ld].view(rows, ld)[:, :width]
    assert view.data_ptr() % 32 == 16
    return view, buf, skip


def _copy_off32(t, ld=None):
    view, _, _ = _off32(t.shape[0], t.shape[1], t.dtype, ld)
    view.copy_(t)
    return view


@pytest.mark.parametrize("table", ["f32", "bf16"])
@pytest.mark.parametrize("out", ["f32", "bf16"])
@pytest.mark.parametrize("T,H", [(1, 8), (3, 264), (257, 1032), (50003, 256)])
def test_lookup(lp, table, out, T, H):
    import torch
    types = {"f32": torch.float32, "bf16": torch.bfloat16}
    V = 1000
    part = lp.VocabPartition(V, V, ((0, 300), (300, V)))
    W = [_normal((300, H), types[table], 1), _normal((700, H), types[table], 2)]
    ids = dev_i32(np.random.RandomState(T).randint(-1, V, T))
    want = lp.lp_embedding(ids, W, part, scale=1.5, out_dtype=types[out])
    moved = [_copy_off32(w) for w in W]
    assert torch.equal(lp.lp_embedding(ids, moved, part, scale=1.5, out_dtype=types[out]), want)
    assert torch.equal(lp.lp_embedding(ids, [W[0], moved[1]], part, scale=1.5, out_dtype=types[out]), want)
    pad = 4 if out == "f32" else 8
    for ld in (H, H + pad):
        y, buf, skip = _off32(T, H, types[out], ld)
        assert lp.lp_embedding(ids, moved, part, scale=1.5, out=y) is y and torch.equal(y, want)
        rows = buf[skip:skip + T * ld].view(T, ld)
        assert bool((buf[:skip] == 5).all()) and bool((buf[skip + T * ld:] == 5).all()) and bool((rows[:, H:] == 5).all())
    # a 32-byte aligned start whose rows' stride is not a multiple of 32 bytes
    y = torch.full((T, H + pad), 5.0, dtype=types[out], device="cuda")[:, :H]
    assert torch.equal(lp.lp_embedding(ids, W, part, scale=1.5, out=y), want)
    assert lp.lp_get_device_error() == 0


@pytest.mark.parametrize("grad", ["bf16", "f32"])
@pytest.mark.parametrize("dw", ["f32", "bf16"])
@pytest.mark.parametrize("T,H", [(60, 264), (600, 8), (3001, 136), (20000, 264)])
def test_gradient(lp, grad, dw, T, H):
    import torch
    types = {"f32": torch.float32, "bf16": torch.bfloat16}
    V, rs = 1000, np.random.RandomState(T)
    part = lp.VocabPartition(V, V, ((0, 300), (300, V)))
    ids = rs.randint(-1, V, T)
    ids[rs.rand(T) < 0.3] = 301                      # a long run
    ids, dY = dev_i32(ids), _normal((T, H), types[grad], 3)
    want = lp.lp_embedding_backward(ids, dY, part, scale=0.5, dw_dtype=types[dw])
    held = [_off32(n, H, types[dw]) for n in (300, 700)]
    pad = 4 if grad == "f32" else 8
    for rows in (dY, _copy_off32(dY), _copy_off32(dY, H + pad)):
        lp.lp_embedding_backward(ids, rows, part, scale=0.5, dw_dtype=types[dw], dW=[v for v, _, _ in held])
        assert all(torch.equal(v, w) for (v, _, _), w in zip(held, want))
    assert all(bool((b[:s] == 5).all()) and bool((b[s + v.numel():] == 5).all()) for v, b, s in held)
    if dw == "f32":
        base = [_normal((n, H), torch.float32, n) for n in (300, 700)]
        for (v, _, _), b in zip(held, base):
            v.copy_(b)
        lp.lp_embedding_backward(ids, dY, part, scale=0.5, accumulate=True, dW=[v for v, _, _ in held])
        assert all(torch.equal(v, b + w) for (v, _, _), b, w in zip(held, base, want))
    assert lp.lp_get_device_error() == 0


def test_autograd_takes_gradients_in_any_order(lp):
    """A transposed, an expanded, a column-sliced and an offset gradient give what their contiguous copies give."""
    import torch
    from lm_head_linear_tcgen05_gb300.autograd import embedding
    V, T, H = 300, 200, 64
    part = lp.VocabPartition(V, V, ((0, 100), (100, V)))
    ids = dev_i32(np.random.RandomState(1).randint(-1, V, T))
    for dtype in (torch.bfloat16, torch.float32):
        W = [_normal((100, H), dtype, 1).requires_grad_(), _normal((200, H), dtype, 2).requires_grad_()]
        D = _normal((T, H), dtype, 3)
        gradients = {
            "transposed": D.t().contiguous().t(), "expanded rows": D[:1].expand(T, H), "expanded": D[0, 0].expand(T, H),
            "sliced": _normal((T, H + 8), dtype, 4)[:, 4:4 + H], "every other": _normal((T, 2 * H), dtype, 5)[:, ::2],
            "odd stride": _normal((T, H + 1), dtype, 6)[:, :H], "reversed": D.flip(0),
        }
        for name, g in gradients.items():
            got = torch.autograd.grad(embedding(ids, W, part, scale=8.0), W, g)
            want = lp.lp_embedding_backward(ids, g.contiguous(), part, scale=8.0, dw_dtype=dtype)
            assert all(torch.equal(a, b) for a, b in zip(got, want)), name
        # as the engine makes it: through a product with the transposed rows
        y, seen = embedding(ids, W, part, scale=8.0), []
        y.register_hook(seen.append)
        (y.t() @ D).float().sum().backward()
        want = lp.lp_embedding_backward(ids, seen[0].contiguous(), part, scale=8.0, dw_dtype=dtype)
        assert all(torch.equal(w.grad, g) for w, g in zip(W, want))
    assert lp.lp_get_device_error() == 0
