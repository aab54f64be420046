"""Refusals of the entry points between the embedding and the losses: the C ABI checks its arguments before any CUDA
work, the binding checks tensors before the call (CPU only; fake, never dereferenced addresses)."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def lp():
    from lm_head_linear_tcgen05_gb300 import _build
    _build.build()
    import lm_head_linear_tcgen05_gb300 as mod
    mod.lib()
    return mod


def _has_gpu():
    import torch
    return torch.cuda.is_available()


no_gpu = pytest.mark.skipif(_has_gpu(), reason="uses fake device pointers; only safe without a GPU")
A = 0x100000
NAN, INF = float("nan"), float("inf")
OK, INVALID, ALIGN, DEVICE, WORKSPACE = 0, 1, 2, 3, 4


def test_packed_structures_have_the_header_s_sizes(lp, tmp_path):
    """And their fields' offsets: the last field of each."""
    cc = shutil.which("gcc") or shutil.which("cc")
    if cc is None:
        pytest.skip("no C compiler")
    forms = {"lp_norm_inputs": (lp._NORM_INPUTS, "ld_gate", 8), "lp_norm_options": (lp._NORM_OPTIONS, "post_norm", 4),
             "lp_norm_outputs": (lp._NORM_OUTPUTS, "ld_norm", 8), "lp_norm_grads": (lp._NORM_GRADS, "accumulate", 4),
             "lp_balance_inputs": (lp._BALANCE_INPUTS, "n_seqs", 8), "lp_balance_options": (lp._BALANCE_OPTIONS, "grad_dtype", 4),
             "lp_balance_outputs": (lp._BALANCE_OUTPUTS, "ld_grad", 8)}
    lines = "".join(f'printf("%zu %zu\\n", sizeof({n}), offsetof({n}, {f}));' for n, (_, f, _) in forms.items())
    src = tmp_path / "s.c"
    src.write_text(f'#include <stdio.h>\n#include <stddef.h>\n#include "lp.h"\nint main(void) {{ {lines} return 0; }}\n')
    subprocess.run([cc, "-I", os.path.join(ROOT, "include"), str(src), "-o", str(tmp_path / "s")], check=True)
    got = subprocess.run([str(tmp_path / "s")], check=True, capture_output=True, text=True).stdout.split("\n")
    for line, (name, (form, _, size)) in zip(got, forms.items()):
        total, last = map(int, line.split())
        pad = total - last - size
        assert total == form.size and (pad == 0 or form.format.endswith(f"{pad}x")), name


@no_gpu
def test_dropout_refuses(lp):
    def call(x=A, T=8, H=64, ld=64, dtype=1, p=0.5, seed=1, offset=0, start=0, rng=None, out=A, ld_out=64):
        return lp.lib().lp_dropout(x, T, H, ld, dtype, p, seed, offset, start, rng, out, ld_out, None)

    assert call() == DEVICE and call(dtype=0, p=0.0, rng=A + 8) == DEVICE and call(start=(1 << 59)) == DEVICE
    for bad in (dict(x=None), dict(out=None), dict(T=-1), dict(H=60), dict(H=0), dict(ld=56), dict(ld_out=56), dict(dtype=2),
                dict(p=-0.1), dict(p=1.1), dict(p=NAN), dict(start=-1), dict(start=(1 << 60) - 4), dict(T=1 << 40)):
        assert call(**bad) == INVALID, bad
    for bad in (dict(x=A + 8), dict(out=A + 4), dict(ld=68), dict(ld_out=68), dict(dtype=0, ld=66), dict(rng=A + 4)):
        assert call(**bad) == ALIGN, bad
    assert call(T=0, x=None, out=None) == OK and call(T=0, p=2.0) == INVALID


INPUTS = dict(h=A, y=A, weight=A, post_weight=None, gate=None, rng=None, ld_h=64, ld_y=64, ld_gate=64)
OPTIONS = dict(eps=1e-6, scale=1.0, wo=0.0, p=0.0, seed=1, offset=0, start=0, h_dtype=1, y_dtype=1, w_dtype=1, kind=0, post=0)

# what the residual norm and its gradient refuse alike
BAD = (dict(h=None), dict(T=-1), dict(H=12), dict(H=0), dict(H=16392), dict(eps=0.0), dict(eps=-1.0), dict(eps=NAN), dict(eps=INF),
       dict(scale=INF), dict(scale=NAN), dict(wo=INF), dict(p=-0.5), dict(p=1.5), dict(p=NAN), dict(start=-1), dict(h_dtype=2),
       dict(y_dtype=-1), dict(w_dtype=3), dict(kind=4), dict(kind=-1), dict(post=2), dict(post_weight=A), dict(kind=1),
       dict(gate=A), dict(ld_h=56), dict(ld_y=56), dict(kind=3, gate=A, ld_gate=56), dict(inputs=None), dict(opts=None))
OFF = (dict(h=A + 8), dict(y=A + 8), dict(weight=A + 8), dict(post=1, post_weight=A + 4), dict(kind=1, gate=A + 8),
       dict(kind=2, gate=A + 2), dict(kind=3, gate=A + 8), dict(ld_h=68), dict(ld_y=68), dict(rng=A + 4),
       dict(h_dtype=0, ld_h=66))


def _packed(lp, kw):
    i = dict(INPUTS, **{k: v for k, v in kw.items() if k in INPUTS})
    o = dict(OPTIONS, **{k: v for k, v in kw.items() if k in OPTIONS})
    ci = None if "inputs" in kw else lp._NORM_INPUTS.pack(*(v or 0 for v in i.values()))
    return ci, None if "opts" in kw else lp._NORM_OPTIONS.pack(*o.values())


@no_gpu
def test_residual_norm_refuses(lp):
    def call(T=8, H=64, h_out=A, norm=A, ld_out=64, ld_norm=64, outputs=True, **kw):
        ci, co = _packed(lp, kw)
        cr = lp._NORM_OUTPUTS.pack(h_out or 0, norm or 0, ld_out, ld_norm) if outputs else None
        return lp.lib().lp_residual_norm(T, H, ci, co, cr, None)

    assert call() == DEVICE and call(norm=None, weight=None) == DEVICE and call(post=1, post_weight=A, kind=2, gate=A + 4) == DEVICE
    assert call(y=None, h_out=None) == DEVICE
    for bad in BAD + (dict(h_out=None), dict(norm=None), dict(outputs=False), dict(ld_out=56), dict(ld_norm=56), dict(y=None),
                      dict(y=None, h_out=None, norm=None, weight=None), dict(y=None, h_out=None, p=0.5),
                      dict(y=None, h_out=None, post=1), dict(y=None, h_out=None, scale=2.0),
                      dict(y=None, h_out=None, kind=2, gate=A)):
        assert call(**bad) == INVALID, bad
    for bad in OFF + (dict(h_out=A + 8), dict(norm=A + 8), dict(ld_out=68), dict(ld_norm=68)):
        assert call(**bad) == ALIGN, bad
    assert call(T=0, h=None, y=None, h_out=None, norm=None) == OK and call(T=0, eps=0.0) == INVALID


@no_gpu
def test_residual_norm_backward_refuses(lp):
    need = lp.lp_norm_workspace_size(1000, 64)
    assert need > 0

    def call(T=1000, H=64, ws=A, wsb=need, grads=True, d_norm=A, d_h_out=A, d_h=A, d_y=A, d_gate=None, d_weight=A, d_post=None,
             ld=(64,) * 5, dw=0, acc=0, **kw):
        ci, co = _packed(lp, kw)
        cg = lp._NORM_GRADS.pack(*(v or 0 for v in (d_norm, d_h_out, d_h, d_y, d_gate, d_weight, d_post)), *ld, dw, acc)
        return lp.lib().lp_residual_norm_backward(T, H, ci, co, cg if grads else None, ws, wsb, None)

    assert call() == DEVICE and call(dw=1) == DEVICE and call(acc=1) == DEVICE and call(d_norm=None, d_weight=None) == DEVICE
    assert call(d_weight=None, ws=None, wsb=0) == DEVICE and call(d_h_out=None) == DEVICE
    assert call(y=None, d_y=None) == DEVICE and call(kind=1, gate=A, d_gate=A) == DEVICE
    for bad in BAD + (dict(grads=False), dict(d_h=None), dict(d_y=None), dict(d_norm=None), dict(d_norm=None, d_h_out=None, d_weight=None),
                      dict(y=None), dict(weight=None), dict(d_post=A), dict(d_gate=A), dict(dw=2), dict(acc=2), dict(acc=1, dw=1),
                      dict(ld=(56, 64, 64, 64, 64)), dict(ld=(64, 56, 64, 64, 64)), dict(ld=(64, 64, 56, 64, 64)),
                      dict(ld=(64, 64, 64, 56, 64)), dict(kind=3, gate=A, d_gate=A, ld=(64, 64, 64, 64, 56))):
        assert call(**bad) == INVALID, bad
    for bad in OFF + (dict(d_norm=A + 8), dict(d_h_out=A + 8), dict(d_h=A + 8), dict(d_y=A + 8), dict(d_weight=A + 2), dict(ws=A + 8),
                      dict(ld=(68, 64, 64, 64, 64)), dict(kind=2, gate=A, d_gate=A + 2), dict(kind=3, gate=A, d_gate=A + 8)):
        assert call(**bad) == ALIGN, bad
    assert call(wsb=need - 1) == WORKSPACE and call(ws=None) == WORKSPACE
    assert call(kind=1, gate=A, d_gate=A, d_weight=None, ws=None) == WORKSPACE and call(T=100, ws=None, wsb=0) == DEVICE
    empty = dict(T=0, h=None, y=None, d_norm=None, d_h_out=None, d_h=None, d_y=None, ws=None, wsb=0)
    assert call(**empty) == DEVICE and call(**empty, acc=1) == OK and call(**dict(empty, d_weight=None)) == OK


@no_gpu
def test_balance_loss_refuses(lp):
    need = lp.lp_balance_workspace_size(100000, 64, 4, 0)
    assert need > 0

    def call(T=100000, E=64, K=4, ws=A, wsb=need, logits=A, ids=A, mask=None, cu=None, up=None, ld=64, S=0, coef=1.0, z=0.0, score=0,
             l_dtype=0, g_dtype=0, metrics=A, experts=A, counts=A, grad=A, ld_g=64, inputs=True, opts=True, outputs=True):
        ci = lp._BALANCE_INPUTS.pack(*(v or 0 for v in (logits, ids, mask, cu, up)), ld, S)
        co, cr = lp._BALANCE_OPTIONS.pack(coef, z, score, l_dtype, g_dtype), lp._BALANCE_OUTPUTS.pack(
            *(v or 0 for v in (metrics, experts, counts, grad)), ld_g)
        return lp.lib().lp_balance_loss(T, E, K, ci if inputs else None, co if opts else None, cr if outputs else None, ws, wsb, None)

    assert call() == DEVICE and call(mask=A + 1, logits=A + 4, ld=65, grad=A + 4) == DEVICE and call(score=1, l_dtype=1, logits=A + 2) == DEVICE
    assert call(grad=None, ld_g=0) == DEVICE and call(T=100, ws=None, wsb=0) == DEVICE
    assert call(cu=A, S=3, wsb=lp.lp_balance_workspace_size(100000, 64, 4, 3)) == DEVICE
    for bad in (dict(inputs=False), dict(opts=False), dict(outputs=False), dict(T=-1), dict(E=0), dict(E=1025), dict(K=0), dict(K=65),
                dict(T=1 << 29), dict(logits=None), dict(ids=None), dict(ld=63), dict(ld_g=63), dict(coef=NAN), dict(coef=INF), dict(z=NAN),
                dict(score=2), dict(score=-1), dict(score=1, z=0.1), dict(l_dtype=2), dict(g_dtype=2), dict(cu=A, S=0), dict(cu=A, S=-1),
                dict(cu=A, S=1 << 25), dict(metrics=None, experts=None, counts=None, grad=None)):
        assert call(**bad) == INVALID, bad
    for bad in (dict(logits=A + 2), dict(ids=A + 2), dict(cu=A + 2, S=1), dict(up=A + 2), dict(metrics=A + 2), dict(experts=A + 4),
                dict(counts=A + 4), dict(grad=A + 2), dict(l_dtype=1, logits=A + 1), dict(ws=A + 8)):
        assert call(**bad) == ALIGN, bad
    assert call(wsb=need - 1) == WORKSPACE and call(ws=None) == WORKSPACE
    assert call(T=0, logits=None, ids=None, ws=None, wsb=0) == DEVICE and call(T=0, coef=NAN) == INVALID


def test_workspace_sizes(lp):
    assert lp.lp_norm_workspace_size(0, 64) == 0 and lp.lp_norm_workspace_size(8, 60) == 0 and lp.lp_norm_workspace_size(8, 16392) == 0
    # a short batch belongs to one cluster, which needs none
    for H, most in ((8, 256), (64, 256), (72, 128), (136, 64), (256, 64), (264, 24), (8192, 24)):
        assert lp.lp_norm_workspace_size(most, H) == 0 and lp.lp_norm_workspace_size(most + 1, H) > 0
    for H in (8, 64, 256, 264, 4096, 8192, 8200, 16384):
        sizes = [lp.lp_norm_workspace_size(T, H) for T in (300, 2000, 10 ** 4, 10 ** 6, 10 ** 9)]
        assert sizes[0] > 0 and sizes == sorted(sizes) and sizes[-1] <= 2 * 4 * H * 152 * 16
    size = lp.lp_balance_workspace_size
    # a short batch runs in one launch, which needs none
    assert size(4096, 64, 8, 0) == 0 and size(100, 64, 8, 20) == 0 and size(10 ** 5, 64, 8, 0) > 0 and size(100, 64, 8, 33) > 0
    assert size(0, 64, 8, 0) == 0 and size(10, 0, 1, 0) == 0 and size(10, 2000, 1, 0) == 0 and size(10, 8, 65, 0) == 0
    assert size(-1, 8, 1, 0) == 0 and size(1 << 29, 8, 4, 0) == 0 and size(10, 8, 1, -1) == 0


def test_the_binding_refuses_host_tensors(lp):
    import torch
    x, ids = torch.zeros(3, 8), torch.zeros(3, 2, dtype=torch.int32)
    for call in (lambda: lp.lp_dropout(x, 0.5, 1), lambda: lp.lp_residual_norm(x, x), lambda: lp.lp_balance_loss(x, ids),
                 lambda: lp.lp_residual_norm_backward(x, x, x)):
        with pytest.raises(TypeError):
            call()


@pytest.mark.parametrize("name", ["upstream", "grads", "metrics", "out", "grad_dtype"])
def test_the_autograd_balance_loss_refuses_what_autograd_gives(name):
    import torch
    from lm_head_linear_tcgen05_gb300.autograd import balance_loss, residual_norm
    with pytest.raises(TypeError):
        balance_loss(torch.zeros(2, 4), torch.zeros(2, 1, dtype=torch.int32), **{name: None})
    with pytest.raises(TypeError):
        residual_norm(torch.zeros(2, 8), out={})
