"""Refusals of the embedding and loss entry points: the C ABI checks its arguments before any CUDA
work, the binding checks tensors before the call (CPU only; fake, never dereferenced addresses)."""
import ctypes

import pytest


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


def _part(lp, real, bounds, local=False):
    return lp._c_partition(lp.VocabPartition(real, bounds[-1], tuple(zip(bounds[:-1], bounds[1:])), local=local))


@no_gpu
def test_embedding_refuses(lp):
    cp, _keep = _part(lp, 1000, [0, 400, 400, 1000])

    def call(ids=A, T=8, H=64, W=(A, None, A), wd=1, scale=1.0, Y=A, ld=64, yd=1, part=cp):
        return lp.lib().lp_embedding(ids, T, H, (ctypes.c_void_p * 3)(*W), wd, ctypes.byref(part), scale, Y, ld, yd,
                                     None)

    assert call() == DEVICE
    assert call(ld=72) == DEVICE and call(wd=0, yd=0, ld=68) == DEVICE
    for bad in (dict(ids=None), dict(T=-1), dict(H=60), dict(H=0), dict(W=(A, None, None)), dict(wd=2), dict(yd=-1),
                dict(scale=NAN), dict(scale=INF), dict(Y=None), dict(ld=56), dict(T=1 << 30, H=65536)):
        assert call(**bad) == INVALID, bad
    for bad in (dict(ids=A + 2), dict(W=(A + 8, None, A)), dict(Y=A + 8), dict(ld=68), dict(yd=0, ld=66)):
        assert call(**bad) == ALIGN, bad
    assert call(T=0, ids=None, W=(None, None, None), Y=None) == OK
    assert call(T=0, scale=NAN) == INVALID
    broken, _keep2 = _part(lp, 1000, [0, 400, 300, 1000])
    assert call(part=broken) == INVALID


@no_gpu
def test_embedding_backward_refuses(lp):
    cp, _keep = _part(lp, 990, [0, 400, 400, 1000])
    need = lp.lib().lp_workspace_size(lp.LP_OP_EMBEDDING_BACKWARD, 100, 64, ctypes.byref(cp))
    assert need > 0

    def call(ids=A, T=100, H=64, dY=A, ld=64, yd=1, scale=1.0, dW=(A, None, A), dw=0, acc=0, ws=A, wsb=need, opts=True):
        o = lp._EmbeddingOptions(dw, acc)
        return lp.lib().lp_embedding_backward(ids, T, H, dY, ld, yd, ctypes.byref(cp), scale, (ctypes.c_void_p * 3)(*dW),
                                              ctypes.byref(o) if opts else None, ws, wsb, None)

    assert call() == DEVICE and call(opts=False) == DEVICE and call(dw=1) == DEVICE and call(acc=1) == DEVICE
    for bad in (dict(ids=None), dict(dY=None), dict(T=-1), dict(H=12), dict(yd=7), dict(dw=2), dict(acc=2), dict(acc=-1),
                dict(acc=1, dw=1), dict(dW=(None, None, A)), dict(ld=60), dict(scale=INF), dict(T=1 << 30, H=65536)):
        assert call(**bad) == INVALID, bad
    for bad in (dict(ids=A + 1), dict(dY=A + 8), dict(ld=68), dict(dW=(A + 4, None, A)), dict(ws=A + 8)):
        assert call(**bad) == ALIGN, bad
    assert call(wsb=need - 1) == WORKSPACE and call(ws=None) == WORKSPACE
    # an empty batch: zeros are written on the device, unless accumulating
    assert call(T=0, ids=None, dY=None, ws=None, wsb=0) == DEVICE
    assert call(T=0, ids=None, dY=None, ws=None, wsb=0, acc=1) == OK


def test_workspace_sizes(lp):
    cp, _keep = _part(lp, 1000, [0, 1000])
    size = lambda T, H=64: lp.lib().lp_workspace_size(lp.LP_OP_EMBEDDING_BACKWARD, T, H, ctypes.byref(cp))  # noqa: E731
    assert size(0) == 0 and size(10, 60) == 0 and 0 < size(10) <= size(1000) <= size(100000)
    for op in (lp.LP_OP_POLICY_LOSS, lp.LP_OP_PREFERENCE_LOSS):
        assert lp.lib().lp_workspace_size(op, 10, 64, ctypes.byref(cp)) == 0
        assert 0 < lp.lp_loss_workspace_size(op, 10 ** 5, 2) <= lp.lp_loss_workspace_size(op, 10 ** 6, 1000)
        # short batches run in one launch, which needs none
        assert lp.lp_loss_workspace_size(op, 16384, 1024) == 0
        assert lp.lp_loss_workspace_size(op, 16385, 2) > 0 and lp.lp_loss_workspace_size(op, 16384, 2050) > 0
        assert lp.lp_loss_workspace_size(op, 0, 2) == 0 and lp.lp_loss_workspace_size(op, -1, 2) == 0
        assert lp.lp_loss_workspace_size(op, 10, -1) == 0
    assert lp.lp_loss_workspace_size(lp.LP_OP_FORWARD, 10, 2) == 0


@no_gpu
def test_policy_loss_refuses(lp):
    need = lp.lp_loss_workspace_size(lp.LP_OP_POLICY_LOSS, 20000, 4)

    def call(T=20000, ws=A, wsb=need, metrics=A, counts=A, g=A, ge=None, **kw):
        i = dict(logp=A, old_logp=A, ref_logp=None, entropy=None, advantages=A, mask=None, cu_seqlens=A, upstream=None,
                 n_seqs=4)
        o = dict(clip_low=0.2, clip_high=0.2, dual_clip=0.0, kl_coef=0.0, entropy_coef=0.0, denominator=0.0,
                 aggregation=1, kl_kind=2, adv_per_seq=0)
        for k, v in kw.items():
            (i if k in i else o)[k] = v
        ci, co, cr = lp._PolicyInputs(**i), lp._PolicyOptions(**o), lp._PolicyOutputs(metrics, counts, g, ge)
        return lp.lib().lp_policy_loss(T, ctypes.byref(ci), ctypes.byref(co), ctypes.byref(cr), ws, wsb, None)

    assert call() == DEVICE and call(clip_low=1.0, dual_clip=1.5, mask=A + 3) == DEVICE
    assert call(aggregation=0, cu_seqlens=None, n_seqs=0) == DEVICE
    for bad in (dict(T=-1), dict(logp=None), dict(old_logp=None), dict(advantages=None), dict(kl_coef=0.1),
                dict(entropy_coef=0.1), dict(ge=A), dict(cu_seqlens=None), dict(aggregation=0, adv_per_seq=1, cu_seqlens=None),
                dict(n_seqs=0), dict(n_seqs=-1), dict(clip_low=-0.1), dict(clip_low=1.5), dict(clip_high=-1.0),
                dict(clip_high=INF), dict(clip_low=NAN), dict(dual_clip=1.0), dict(dual_clip=-2.0), dict(dual_clip=NAN),
                dict(kl_coef=NAN), dict(entropy_coef=INF), dict(denominator=-1.0), dict(denominator=NAN),
                dict(aggregation=3), dict(kl_kind=3), dict(adv_per_seq=2), dict(metrics=None, counts=None, g=None)):
        assert call(**bad) == INVALID, bad
    for bad in (dict(logp=A + 2), dict(ref_logp=A + 1), dict(cu_seqlens=A + 2), dict(g=A + 2), dict(metrics=A + 1),
                dict(counts=A + 4), dict(upstream=A + 3), dict(ws=A + 8)):
        assert call(**bad) == ALIGN, bad
    assert call(wsb=need - 1) == WORKSPACE and call(ws=None) == WORKSPACE
    assert call(T=100, ws=None, wsb=0) == DEVICE
    assert call(T=0, logp=None, ws=None, wsb=0) == DEVICE and call(T=0, clip_low=-1.0) == INVALID


@no_gpu
def test_preference_loss_refuses(lp):
    need = lp.lp_loss_workspace_size(lp.LP_OP_PREFERENCE_LOSS, 20000, 4)

    def call(T=20000, ws=A, wsb=need, metrics=A, counts=A, h=A, g=A, **kw):
        i = dict(logp=A, ref_logp=None, mask=None, cu_seqlens=A, upstream=None, n_pairs=2)
        o = dict(beta=0.1, label_smoothing=0.0, margin=0.0, denominator=0.0, kind=0, length_normalised=0)
        for k, v in kw.items():
            (i if k in i else o)[k] = v
        ci, co, cr = lp._PreferenceInputs(**i), lp._PreferenceOptions(**o), lp._PreferenceOutputs(metrics, counts, h, g)
        return lp.lib().lp_preference_loss(T, ctypes.byref(ci), ctypes.byref(co), ctypes.byref(cr), ws, wsb, None)

    assert call() == DEVICE and call(label_smoothing=0.3, margin=-1.0) == DEVICE
    for bad in (dict(T=-1), dict(logp=None), dict(cu_seqlens=None), dict(n_pairs=0), dict(n_pairs=-1),
                dict(n_pairs=1 << 30), dict(beta=0.0), dict(beta=-1.0), dict(beta=NAN), dict(label_smoothing=1.0),
                dict(label_smoothing=-0.1), dict(kind=1, label_smoothing=0.1), dict(kind=3), dict(margin=NAN),
                dict(length_normalised=2), dict(denominator=-1.0), dict(metrics=None, counts=None, h=None, g=None)):
        assert call(**bad) == INVALID, bad
    for bad in (dict(logp=A + 2), dict(g=A + 1), dict(h=A + 2), dict(counts=A + 4), dict(ws=A + 4)):
        assert call(**bad) == ALIGN, bad
    assert call(wsb=need - 1) == WORKSPACE and call(T=100, ws=None, wsb=0) == DEVICE
    assert call(T=0, logp=None, ws=None, wsb=0) == DEVICE


def test_the_binding_refuses_host_tensors(lp):
    import torch
    part = lp.VocabPartition(10, 10, ((0, 10),))
    ids, W, x, cu = torch.zeros(3, dtype=torch.int32), torch.zeros(10, 8), torch.zeros(3), torch.zeros(3, dtype=torch.int32)
    with pytest.raises(ValueError):
        lp.lp_embedding(ids, [W], part)
    with pytest.raises(ValueError):
        lp.lp_embedding_backward(ids, torch.zeros(3, 8), part)
    with pytest.raises(ValueError):
        lp.lp_policy_loss(x, x, x)
    with pytest.raises(ValueError):
        lp.lp_preference_loss(x, cu)
