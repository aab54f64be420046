"""A training step of a small policy with routed experts' loads, from the token ids to two losses and back, through the
operators in the order of their use, against the same step in 64 bits.

The step rounds to bf16 in a dozen places between a parameter and its gradient (the embedded rows, each norm, each
block output, the head's input, their gradients on the way back), each by at most 2^-8 and 2^-8 / sqrt(3) in the root
mean square: errors of unlike sign add up to sqrt(12) 2^-8 / sqrt(3) = 0.008 of a gradient's norm, and twice that where
two paths meet. 0.03 leaves twice that."""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
import block_ref as ref  # noqa: E402

T, H, V, E, K = 160, 64, 320, 8, 2
BF = torch.bfloat16


@pytest.fixture(scope="module")
def lp():
    from lm_head_linear_tcgen05_gb300 import _build
    _build.build()
    import lm_head_linear_tcgen05_gb300 as mod
    torch.cuda.set_device(0)
    return mod


def parameters():
    gen = torch.Generator(device="cuda").manual_seed(1)
    n = lambda *s, std=1.0, mean=0.0, dt=BF: torch.empty(s, dtype=dt, device="cuda").normal_(mean, std, generator=gen).requires_grad_()  # noqa: E731
    P = dict(table=n(V, H), head=n(V, H, std=0.1), final=n(H, std=0.1, mean=1.0))
    for b in range(2):
        P.update({f"mix{b}": n(H, H, std=0.15), f"router{b}": n(E, H, std=0.2), f"norm{b}": n(H, std=0.1, mean=1.0),
                  f"post{b}": n(H, std=0.1, mean=1.0), f"gate{b}": n(H, std=0.1, mean=0.7)})
    ids = torch.randint(0, V, (T,), device="cuda", generator=gen, dtype=torch.int32)
    y = torch.randint(0, V, (T,), device="cuda", generator=gen, dtype=torch.int32)
    adv = torch.randn(T, device="cuda", generator=gen)
    mask = (torch.rand(T, device="cuda", generator=gen) < 0.8).to(torch.uint8)
    return P, ids, y, adv, mask


def step(lp, P, ids, y, adv, mask, cu):
    from lm_head_linear_tcgen05_gb300 import autograd as A
    part = lp.VocabPartition(V, V, ((0, V),))
    h = A.dropout(A.embedding(ids, [P["table"]], part, out_dtype=torch.float32), 0.1, 7)
    _, x = A.residual_norm(h, weight=P["norm0"], norm_dtype=BF)
    loss, chosen = 0.0, []
    for b in range(2):
        logits = (x @ P[f"router{b}"].t()).float()
        experts = logits.detach().topk(K, 1).indices.to(torch.int32)
        chosen.append(experts)
        out = A.balance_loss(logits, experts, coef=0.1, z_coef=0.01, mask=mask, cu_seqlens=cu)
        loss = loss + out[0]
        y_block = torch.nn.functional.silu(x @ P[f"mix{b}"].t())
        h, x = A.residual_norm(h, y_block, weight=P["norm1"] if b == 0 else P["final"], post_norm=True, post_weight=P[f"post{b}"],
                               gate=P[f"gate{b}"], dropout=0.1, seed=7, offset=1 + b)
    logp, _ = A.linear_logp(x, [P["head"]], None, part, y, 1.0)
    policy, _, _ = A.policy_loss(logp, logp.detach(), adv, mask=mask)
    return loss + policy, chosen


def plain_step(P, ids, y, adv, mask, cu, chosen):
    h = P["table"][ids.long()]
    keep, f = ref.kept(T, H, 0.1, 7, 0, 0, "cuda")
    h = torch.where(keep, h * f, 0.0)
    x = ref.norm(h, weight=P["norm0"])[1]
    loss, kept = 0.0, mask.double()
    for b in range(2):
        l = x @ P[f"router{b}"].t()
        w, share = torch.zeros_like(l), torch.zeros_like(l)
        c = cu.tolist() if cu is not None else [0, T]
        live = sum(int(mask[a:z].sum()) > 0 for a, z in zip(c[:-1], c[1:]))
        for a, z in zip(c[:-1], c[1:]):
            n = max(int(mask[a:z].sum()), 1)
            used = chosen[b][a:z][mask[a:z] != 0].reshape(-1).long()
            share[a:z] = torch.bincount(used, minlength=E).double() * E / (K * n)
            w[a:z] = 1.0 / (n * live)
        p = torch.softmax(l, 1)
        loss = loss + 0.1 * (kept[:, None] * w * share * p).sum() + 0.01 * (kept * torch.logsumexp(l, 1) ** 2).sum() / kept.sum()
        block = torch.nn.functional.silu(x @ P[f"mix{b}"].t())
        h, x, _, _ = ref.norm(h, block, weight=P["norm1"] if b == 0 else P["final"], post_norm=True, post_weight=P[f"post{b}"],
                              gate=P[f"gate{b}"], dropout=0.1, seed=7, offset=1 + b)
    logp = torch.log_softmax(x @ P["head"].t(), 1).gather(1, y.long()[:, None])[:, 0]
    return loss - (kept * adv.double() * torch.exp(logp - logp.detach())).sum() / kept.sum()


@pytest.mark.parametrize("cu", [None, [0, 50, 50, 120, T]])
def test_a_step(lp, cu):
    P, ids, y, adv, mask = parameters()
    cu = None if cu is None else torch.tensor(cu, dtype=torch.int32, device="cuda")
    loss, chosen = step(lp, P, ids, y, adv, mask, cu)
    grads = torch.autograd.grad(loss, list(P.values()))
    again = torch.autograd.grad(step(lp, P, ids, y, adv, mask, cu)[0], list(P.values()))
    wide = {k: v.detach().double().requires_grad_() for k, v in P.items()}
    want = plain_step(wide, ids, y, adv, mask, cu, chosen)
    expected = torch.autograd.grad(want, list(wide.values()))
    assert abs(float(loss.detach()) - float(want.detach())) < 0.03 * (1 + abs(float(want.detach())))
    for k, g, g2, e in zip(P, grads, again, expected):
        assert torch.equal(g, g2), k
        error = float((g.double() - e).norm() / e.norm())
        assert error < 0.03, (k, error)
    assert lp.lp_get_device_error() == 0


def test_a_step_in_a_graph(lp):
    """The same calls captured once (forward and backward of the entry points themselves) and replayed."""
    P, ids, y, adv, mask = parameters()
    P = {k: v.detach() for k, v in P.items()}
    part = lp.VocabPartition(V, V, ((0, V),))
    rng = torch.zeros(2, dtype=torch.int64, device="cuda")
    o = dict(weight=P["final"], post_norm=True, post_weight=P["post0"], gate=P["gate0"], dropout=0.1, seed=7, rng=rng)

    def run():
        h = lp.lp_dropout(lp.lp_embedding(ids, [P["table"]], part), 0.1, 7, offset=9, rng=rng)
        x = lp.lp_residual_norm(h, weight=P["norm0"])[1]
        logits = x @ P["router0"].t()
        balance = lp.lp_balance_loss(logits, logits.topk(K, 1).indices.to(torch.int32), mask=mask)
        block = x @ P["mix0"].t()
        h_out, x = lp.lp_residual_norm(h, block, **o)
        out = lp.lp_forward(x, [P["head"]], None, part, y, 1.0)
        g = lp.lp_backward(x, [P["head"]], None, part, y, 1.0, out["lse"], adv)
        d = lp.lp_residual_norm_backward(h_out, block, g["dX"].to(BF), None, **o)
        return [out["logp"], balance["metrics"], balance["grad_logits"], *[v for v in d.values() if v is not None]]

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        run()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            got = run()
    torch.cuda.current_stream().wait_stream(s)
    first = None
    for i in (1, 2):
        rng[1] = 100 * i
        graph.replay()
        for a, b in zip(got, run()):
            assert torch.equal(a, b)
        first = got[0].clone() if first is None else first
    assert not torch.equal(first, got[0])          # other bits were drawn
    assert lp.lp_get_device_error() == 0
