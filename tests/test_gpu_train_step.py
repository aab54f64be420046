"""The embedding and the losses as they are used: the autograd wrappers, a whole step with a table
tied to the head, the example; and the checks that stand in for a sanitizer: canary words around
every buffer, the bounds-checked build, refusals of tensors that do not fit."""
import ctypes
import math
import os
import sys

import numpy as np
import pytest

from lp_util import dev_f32, dev_i32, rel_fro
from oracle import train

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def lp():
    from lm_head_linear_tcgen05_gb300 import _build
    _build.build()
    import lm_head_linear_tcgen05_gb300 as mod
    import torch
    assert mod.lp_device_supported()
    torch.cuda.set_device(0)
    return mod


def _normal(shape, dtype, seed, std=1.0):
    import torch
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return torch.empty(shape, dtype=dtype, device="cuda").normal_(0.0, std, generator=g)


def test_autograd_gradients_are_the_library_calls(lp):
    import torch
    from lm_head_linear_tcgen05_gb300.autograd import embedding, policy_loss, preference_loss
    part = lp.VocabPartition(300, 304, ((0, 100), (100, 304)))
    rs = np.random.RandomState(0)
    ids = dev_i32(rs.randint(-1, 300, 200))
    W = [_normal((100, 64), torch.bfloat16, 1).requires_grad_(), _normal((204, 64), torch.bfloat16, 2).requires_grad_()]
    dY = _normal((200, 64), torch.bfloat16, 3)
    y = embedding(ids, W, part, scale=8.0)
    y.backward(dY)
    want = lp.lp_embedding_backward(ids, dY, part, scale=8.0, dw_dtype=torch.bfloat16)
    assert all(torch.equal(w.grad, g) for w, g in zip(W, want))
    for w in W:
        w.grad = None
    embedding(ids, W, part, scale=8.0).sum().backward()       # an expanded gradient, every stride zero
    want = lp.lp_embedding_backward(ids, torch.ones_like(dY), part, scale=8.0, dw_dtype=torch.bfloat16)
    assert all(torch.equal(w.grad, g) for w, g in zip(W, want))
    W[1].grad = None
    (embedding(ids, W, part).t() @ dY.float().to(torch.bfloat16)).float().sum().backward()   # a transposed one
    assert bool(W[1].grad.isfinite().all())

    logp, old, ref = dev_f32(-rs.rand(200)), dev_f32(-rs.rand(200)), dev_f32(-rs.rand(200))
    ent, adv, cu = dev_f32(rs.rand(200)), dev_f32(rs.randn(4)), dev_i32([0, 50, 50, 120, 200])
    mask = torch.from_numpy(rs.rand(200) < 0.8).cuda()
    opts = dict(ref_logp=ref, mask=mask, cu_seqlens=cu, kl_coef=0.1, entropy_coef=0.2, aggregation="seq_mean_token_mean")
    a, b = logp.clone().requires_grad_(), ent.clone().requires_grad_()
    loss, metrics, counts = policy_loss(a, old, adv, entropy=b, **opts)
    (3.0 * loss).backward()
    direct = lp.lp_policy_loss(logp, old, adv, entropy=ent, upstream=torch.tensor(3.0, device="cuda"), **opts)
    assert torch.equal(a.grad, direct["grad_logp"]) and torch.equal(b.grad, direct["grad_entropy"])
    assert torch.equal(metrics, direct["metrics"]) and float(loss.detach()) == float(direct["loss"])
    assert torch.equal(counts, direct["counts"])
    a = logp.clone().requires_grad_()
    loss, _, _, margins = preference_loss(a, cu, ref_logp=ref, mask=mask, beta=0.5)
    (-loss).backward()
    direct = lp.lp_preference_loss(logp, cu, ref_logp=ref, mask=mask, beta=0.5,
                                   upstream=torch.tensor(-1.0, device="cuda"))
    assert torch.equal(a.grad, direct["grad_logp"]) and torch.equal(margins, direct["margins"])
    assert lp.lp_get_device_error() == 0


def test_autograd_notices_inputs_changed_in_place(lp):
    # the backward reads the inputs again: one that was changed since must not be used in silence
    import torch
    from lm_head_linear_tcgen05_gb300.autograd import embedding, policy_loss, preference_loss
    rs = np.random.RandomState(5)
    cu, old = dev_i32([0, 30, 64]), dev_f32(-rs.rand(64))
    for name in ("mask", "ref_logp", "old_logp", "advantages", "entropy", "cu_seqlens"):
        logp = dev_f32(-rs.rand(64)).requires_grad_()
        args = {"old_logp": old.clone(), "advantages": dev_f32(rs.randn(64)), "entropy": dev_f32(rs.rand(64)),
                "ref_logp": old.clone(), "mask": torch.ones(64, dtype=torch.bool, device="cuda"),
                "cu_seqlens": cu.clone()}
        loss, *_ = policy_loss(logp, kl_coef=0.1, aggregation="seq_mean_token_mean", **args)
        args[name].zero_()
        with pytest.raises(RuntimeError, match="modified by an inplace operation"):
            loss.backward()
    for name in ("mask", "ref_logp", "cu_seqlens"):
        logp = dev_f32(-rs.rand(64)).requires_grad_()
        args = {"ref_logp": old.clone(), "mask": torch.ones(64, dtype=torch.bool, device="cuda"),
                "cu_seqlens": cu.clone()}
        loss, *_ = preference_loss(logp, **args)
        args[name].zero_()
        with pytest.raises(RuntimeError, match="modified by an inplace operation"):
            loss.backward()
    ids, W = dev_i32(rs.randint(0, 50, 9)), _normal((50, 16), torch.float32, 1).requires_grad_()
    y = embedding(ids, [W], lp.VocabPartition(50, 50, ((0, 50),)))
    ids.zero_()
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        y.sum().backward()


def test_autograd_refuses_second_derivatives(lp):
    import torch
    from lm_head_linear_tcgen05_gb300.autograd import preference_loss
    rs = np.random.RandomState(6)
    logp = dev_f32(-rs.rand(64)).requires_grad_()
    loss, *_ = preference_loss(logp, dev_i32([0, 30, 64]))
    (g,) = torch.autograd.grad(loss * logp.sum(), logp, create_graph=True)
    with pytest.raises(RuntimeError, match="once_differentiable"):
        g.sum().backward()


def test_tied_table_step_matches_fp64(lp):
    """lookup -> linear-logp -> policy loss -> backward -> the lookup's gradient added to the head's:
    the table's whole gradient against fp64 autograd of the same function (X rounded to bf16 alike)."""
    import torch
    V, H, T = 500, 128, 300
    rs = np.random.RandomState(1)
    part = lp.VocabPartition(V, 512, ((0, 256), (256, 512)))
    full = _normal((512, H), torch.bfloat16, 4, 0.2)
    W = [full[:256].contiguous(), full[256:].contiguous()]
    ids, y = dev_i32(rs.randint(-1, V, T)), dev_i32(rs.randint(0, V, T))
    cu, adv = dev_i32([0, 100, 100, 170, 300]), dev_f32(rs.randn(4))
    mask = torch.from_numpy(rs.rand(T) < 0.7).cuda()
    X = lp.lp_embedding(ids, W, part, scale=2.0)
    out = lp.lp_forward(X, W, None, part, y, 0.8)
    old = out["logp"] + 0.05 * _normal(T, torch.float32, 9)
    opts = dict(mask=mask, cu_seqlens=cu, entropy_coef=0.01, aggregation="seq_mean_token_sum")
    loss = lp.lp_policy_loss(out["logp"], old, adv, entropy=out["entropy"], **opts)
    g = lp.lp_backward_ex(X, W, None, part, y, 0.8, out["lse"], loss["grad_logp"], bias_grad=False,
                          entropy=out["entropy"], grad_entropy=loss["grad_entropy"])
    lp.lp_embedding_backward(ids, g["dX"], part, scale=2.0, accumulate=True, dW=g["dW"])

    table = full[:V].double().cpu().requires_grad_()
    used = (ids >= 0).cpu()
    x = torch.where(used[:, None], 2.0 * table[ids.clamp(min=0).long().cpu()], 0.0)
    x = x + (X.double().cpu() - x).detach()                                  # the rounding of X
    p = torch.log_softmax(x @ table.T / 0.8, dim=1)
    lg, ent = p[torch.arange(T), y.long().cpu()], -(p.exp() * p).sum(dim=1)
    ref = train.policy_loss(lg.detach().numpy(), old.double().cpu().numpy(), adv.cpu().numpy(),
                            entropy=ent.detach().numpy(), mask=mask.cpu().numpy(), cu=cu.cpu().numpy(),
                            entropy_coef=0.01, aggregation="seq_mean_token_sum", per_seq=True)
    (lg * torch.from_numpy(ref["grad_logp"]) + ent * torch.from_numpy(ref["grad_entropy"])).sum().backward()
    got = torch.cat(g["dW"])
    assert rel_fro(got[:V].cpu().numpy(), table.grad.numpy()) <= 1e-2      # G is rounded to bf16 inside lp_backward
    assert torch.count_nonzero(got[V:]) == 0
    assert abs(float(loss["loss"]) - ref["metrics"][0]) <= 2e-3 * (1 + ref["mag"][0])
    assert lp.lp_get_device_error() == 0


@pytest.mark.parametrize("objective", ["policy", "preference"])
def test_example_learns(lp, objective):
    sys.path.insert(0, os.path.join(ROOT, "examples"))
    try:
        import tied_policy_step
    finally:
        sys.path.pop(0)
    losses = tied_policy_step.train(steps=12, objective=objective)
    assert all(math.isfinite(x) for x in losses) and losses[-1] < losses[0]
    assert losses == tied_policy_step.train(steps=12, objective=objective)     # the same bits again


CANARY, GUARD = 0x7FC0DEAD, 1024


class _Guarded:
    """`nbytes` of device memory between canary words."""

    def __init__(self, nbytes, fill=None):
        import torch
        self.words = (nbytes + 3) // 4
        self.buf = torch.full((self.words + 2 * GUARD,), CANARY, dtype=torch.int32, device="cuda")
        if fill is not None:
            self.buf[GUARD:GUARD + self.words] = fill
        self.nbytes, self.ptr = nbytes, self.buf.data_ptr() + 4 * GUARD

    def intact(self):
        raw = self.buf.cpu().numpy().view(np.uint8)
        want = np.full(GUARD, CANARY, dtype=np.uint32).view(np.uint8)
        tail = 4 * GUARD + self.nbytes
        pattern = np.full(self.words + 2 * GUARD, CANARY, dtype=np.uint32).view(np.uint8)
        return bool(np.array_equal(raw[:4 * GUARD], want) and np.array_equal(raw[tail:], pattern[tail:]))


@pytest.mark.parametrize("T,H,hot", [(1, 8, 0.0), (333, 264, 0.6), (20000, 72, 0.5)])
@pytest.mark.parametrize("acc,dw", [(0, 0), (0, 1), (1, 0)])
def test_embedding_writes_only_inside_its_buffers(lp, T, H, hot, acc, dw):
    import torch
    L = lp.lib()
    rs = np.random.RandomState(T)
    cp, _keep = lp._c_partition(lp.VocabPartition(1000, 1024, ((0, 300), (300, 300), (300, 1024))))
    ids = rs.randint(-1, 1000, T)
    ids[rs.rand(T) < hot] = 301
    ids = dev_i32(ids)
    W = [_normal((n, H), torch.bfloat16, n) for n in (300, 724)]
    Y = _Guarded(T * H * 2)
    Wp = (ctypes.c_void_p * 3)(W[0].data_ptr(), None, W[1].data_ptr())
    assert L.lp_embedding(ids.data_ptr(), T, H, Wp, 1, ctypes.byref(cp), 1.5, Y.ptr, H, 1, None) == 0
    dY = _normal((T, H), torch.bfloat16, 5)
    ws = _Guarded(L.lp_workspace_size(lp.LP_OP_EMBEDDING_BACKWARD, T, H, ctypes.byref(cp)))
    dW = [_Guarded(n * H * (2 if dw else 4), 0 if acc else None) for n in (300, 724)]
    dWp = (ctypes.c_void_p * 3)(dW[0].ptr, None, dW[1].ptr)
    o = lp._EmbeddingOptions(dw, acc)
    assert L.lp_embedding_backward(ids.data_ptr(), T, H, dY.data_ptr(), H, 1, ctypes.byref(cp), 1.5, dWp,
                                   ctypes.byref(o), ws.ptr, ws.nbytes, None) == 0
    torch.cuda.synchronize()
    assert all(b.intact() for b in (Y, ws, *dW))
    assert lp.lp_get_device_error() == 0


@pytest.mark.parametrize("T,S", [(1, 2), (1001, 16), (20001, 400), (70003, 6)])
def test_losses_write_only_inside_their_buffers(lp, T, S):
    import torch
    L = lp.lib()
    rs = np.random.RandomState(T)
    cu = dev_i32(np.sort(np.concatenate([[0, T], rs.randint(0, T + 1, S - 1)])))
    x = dev_f32(-rs.rand(T))
    for offset in (0, 4):            # the outputs 16- and 4-byte aligned
        m, c, g, ge, h = _Guarded(24), _Guarded(16), _Guarded(4 * T + offset), _Guarded(4 * T + offset), _Guarded(2 * S)
        ws = _Guarded(lp.lp_loss_workspace_size(lp.LP_OP_POLICY_LOSS, T, S))
        i = lp._PolicyInputs(x.data_ptr(), x.data_ptr(), x.data_ptr(), x.data_ptr(), x.data_ptr(), None, cu.data_ptr(),
                             None, S)
        o = lp._PolicyOptions(0.2, 0.2, 0.0, 0.1, 0.1, 0.0, 1, 2, 0)
        r = lp._PolicyOutputs(m.ptr, c.ptr, g.ptr + offset, ge.ptr + offset)
        assert L.lp_policy_loss(T, ctypes.byref(i), ctypes.byref(o), ctypes.byref(r), ws.ptr, ws.nbytes, None) == 0
        ws2 = _Guarded(lp.lp_loss_workspace_size(lp.LP_OP_PREFERENCE_LOSS, T, S))
        m2, c2, g2 = _Guarded(20), _Guarded(8), _Guarded(4 * T + offset)
        i = lp._PreferenceInputs(x.data_ptr(), None, None, cu.data_ptr(), None, S // 2)
        o = lp._PreferenceOptions(0.1, 0.0, 0.0, 0.0, 0, 0)
        r = lp._PreferenceOutputs(m2.ptr, c2.ptr, h.ptr, g2.ptr + offset)
        assert L.lp_preference_loss(T, ctypes.byref(i), ctypes.byref(o), ctypes.byref(r), ws2.ptr, ws2.nbytes, None) == 0
        torch.cuda.synchronize()
        assert all(b.intact() for b in (m, c, g, ge, h, ws, ws2, m2, c2, g2))
    assert lp.lp_get_device_error() == 0


def test_bounds_checked_build_gives_the_same_bits(lp):
    import torch
    from lm_head_linear_tcgen05_gb300 import _build
    regular, debug = _build.build(), _build.build(debug_bounds=True)
    part = lp.VocabPartition(8100, 8192, ((0, 3000), (3000, 3000), (3000, 8192)))
    rs = np.random.RandomState(3)
    T, H = 17000, 136
    ids = rs.randint(-1, 8100, T)
    ids[rs.rand(T) < 0.3] = 5
    ids, dY = dev_i32(ids), _normal((T, H), torch.float32, 1)
    W = [_normal((3000, H), torch.float32, 2), None, _normal((5192, H), torch.float32, 3)]
    x, old = dev_f32(-rs.rand(T)), dev_f32(-rs.rand(T))
    cu = dev_i32([0, 10, 10, 9000, T])

    def calls():
        p = lp.lp_policy_loss(x, old, old, ref_logp=old, kl_coef=0.1, cu_seqlens=cu, aggregation="seq_mean_token_mean")
        q = lp.lp_preference_loss(x, cu, ref_logp=old)
        return [lp.lp_embedding(ids, W, part, scale=3.0, out_dtype=torch.bfloat16),
                *[d for d in lp.lp_embedding_backward(ids, dY, part) if d is not None],
                p["metrics"], p["grad_logp"], q["metrics"], q["grad_logp"]]

    lp.use_library(regular)
    want = calls()
    try:
        lp.use_library(debug)
        got = calls()
        assert lp.lp_get_device_error() == 0
    finally:
        lp.use_library(regular)
    assert all(torch.equal(a, b) for a, b in zip(want, got))


def test_the_binding_refuses_tensors_that_do_not_fit(lp):
    import torch
    part = lp.VocabPartition(100, 100, ((0, 100),))
    ids, W, dY = dev_i32(np.zeros(6)), _normal((100, 16), torch.bfloat16, 1), _normal((6, 16), torch.bfloat16, 2)
    x, cu = torch.zeros(6, device="cuda"), dev_i32([0, 2, 6])
    bad = [
        lambda: lp.lp_embedding(ids.long(), [W], part),
        lambda: lp.lp_embedding(ids, [W.half()], part),
        lambda: lp.lp_embedding(ids, [W[:50]], part),
        lambda: lp.lp_embedding(ids, [W, W], part),
        lambda: lp.lp_embedding(ids, [W.t().contiguous().t()], part),
        lambda: lp.lp_embedding(ids, [W], part, out_dtype=torch.float16),
        lambda: lp.lp_embedding(ids, [W], part, out=torch.empty(6, 24, dtype=torch.bfloat16, device="cuda")),
        lambda: lp.lp_embedding(ids, [W], part, out=torch.empty(16, 6, dtype=torch.bfloat16, device="cuda").t()),
        lambda: lp.lp_embedding_backward(ids, dY[:5], part),
        lambda: lp.lp_embedding_backward(ids, dY.t().contiguous().t(), part),
        lambda: lp.lp_embedding_backward(ids, dY, part, accumulate=True),
        lambda: lp.lp_embedding_backward(ids, dY, part, accumulate=True, dw_dtype=torch.bfloat16, dW=[W]),
        lambda: lp.lp_embedding_backward(ids, dY, part, dW=[torch.empty(99, 16, device="cuda")]),
        lambda: lp.lp_embedding_backward(ids, dY, part, workspace=torch.empty(16, dtype=torch.uint8, device="cuda")),
        lambda: lp.lp_policy_loss(x, x[:5], x),
        lambda: lp.lp_policy_loss(x, x, x[:2].contiguous()),
        lambda: lp.lp_policy_loss(x, x, x[:2].contiguous(), adv_per_seq=True),
        lambda: lp.lp_policy_loss(x, x, x, mask=x),
        lambda: lp.lp_policy_loss(x, x, x, aggregation="mean"),
        lambda: lp.lp_policy_loss(x, x, x, aggregation="seq_mean_token_sum"),
        lambda: lp.lp_policy_loss(x, x, x, kl_coef=0.1),
        lambda: lp.lp_policy_loss(x, x, x, clip_low=2.0),
        lambda: lp.lp_policy_loss(x, x, x, upstream=torch.ones(2, device="cuda")),
        lambda: lp.lp_policy_loss(x, x, x, upstream=torch.ones(1)),
        lambda: lp.lp_policy_loss(x.double(), x, x),
        lambda: lp.lp_policy_loss(torch.zeros(12, device="cuda")[::2], x, x),
        lambda: lp.lp_preference_loss(x, cu[:2].contiguous()),
        lambda: lp.lp_preference_loss(x, cu.long()),
        lambda: lp.lp_preference_loss(x, cu, kind="dpo"),
        lambda: lp.lp_preference_loss(x, cu, beta=0.0),
        lambda: lp.lp_preference_loss(x, cu, kind="ipo", label_smoothing=0.1),
    ]
    for f in bad:
        with pytest.raises((TypeError, ValueError, RuntimeError)):
            f()
    assert lp.lp_get_device_error() == 0


def test_the_binding_refuses_workspaces_that_do_not_fit(lp):
    # every call refuses before anything is launched
    import torch
    T = 20000
    part = lp.VocabPartition(100, 100, ((0, 100),))
    ids, dY, x = dev_i32(np.zeros(T)), torch.zeros((T, 16), device="cuda"), torch.zeros(T, device="cuda")
    cu = dev_i32([0, 3, T])
    n = 1 << 22
    assert lp.lp_loss_workspace_size(lp.LP_OP_POLICY_LOSS, T, 2) > 0
    assert lp.lp_loss_workspace_size(lp.LP_OP_PREFERENCE_LOSS, T, 2) > 0
    for ws in (torch.empty(n, dtype=torch.uint8), torch.empty(2 * n, dtype=torch.uint8, device="cuda")[::2],
               torch.empty(16, dtype=torch.uint8, device="cuda"), n):
        for call in (lambda: lp.lp_embedding_backward(ids, dY, part, workspace=ws),
                     lambda: lp.lp_policy_loss(x, x, x, cu_seqlens=cu, workspace=ws),
                     lambda: lp.lp_preference_loss(x, cu, workspace=ws)):
            with pytest.raises((TypeError, ValueError, RuntimeError)):
                call()
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    assert lp.lp_policy_loss(x, x, x, cu_seqlens=cu, workspace=ws)["counts"].tolist() == [T, 2]
    assert lp.lp_get_device_error() == 0


def test_back_to_back_calls_repeat_their_bits(lp):
    """Calls of two inputs in turn, nothing waiting in between: every result is that of the first call."""
    import torch
    part = lp.VocabPartition(5000, 5120, ((0, 2000), (2000, 5120)))
    sets = []
    for seed, T in ((1, 18000), (2, 701)):
        rs = np.random.RandomState(seed)
        ids = rs.randint(-1, 5000, T)
        ids[rs.rand(T) < 0.4] = 7
        cu = np.sort(np.concatenate([[0, T], rs.randint(0, T + 1, 31)]))
        sets.append((dev_i32(ids), _normal((T, 136), torch.bfloat16, seed), dev_f32(-rs.rand(T)), dev_f32(-rs.rand(T)),
                     dev_i32(cu), torch.from_numpy(rs.rand(T) < 0.7).cuda()))

    def calls(s):
        ids, dY, x, old, cu, mask = s
        g = lp.lp_embedding_backward(ids, dY, part, scale=0.5)
        lp.lp_embedding_backward(ids, dY, part, accumulate=True, dW=g)
        p = lp.lp_policy_loss(x, old, old, ref_logp=old, entropy=old, mask=mask, cu_seqlens=cu, kl_coef=0.1,
                              entropy_coef=0.1, aggregation="seq_mean_token_mean")
        q = lp.lp_preference_loss(x, cu, ref_logp=old, mask=mask)
        return [*g, *(p[k] for k in ("metrics", "counts", "grad_logp", "grad_entropy")),
                *(q[k] for k in ("metrics", "margins", "grad_logp"))]

    want = [calls(s) for s in sets]
    for _ in range(12):
        got = [calls(sets[i % 2]) for i in range(10)]
        assert all(torch.equal(a, b) for i, g in enumerate(got) for a, b in zip(g, want[i % 2]))
    assert lp.lp_get_device_error() == 0
