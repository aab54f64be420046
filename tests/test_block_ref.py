"""The 64-bit definitions that the GPU tests compare with: the generator's published vectors, gradients against
automatic differentiation and against differences (CPU only)."""
import pytest
import torch

import block_ref as ref


def test_the_generator_gives_the_published_vectors():
    assert ref.philox([0] * 4, [0] * 2) == [0x6627E8D5, 0xE169C58D, 0xBC57AC4C, 0x9B00DBD8]
    assert ref.philox([0xFFFFFFFF] * 4, [0xFFFFFFFF] * 2) == [0x408F276D, 0x41C83B0E, 0xA20BC7C6, 0x6D5451FD]
    assert ref.philox([0x243F6A88, 0x85A308D3, 0x13198A2E, 0x03707344], [0xA4093822, 0x299F31D0]) == [
        0xD16CFE09, 0x94FDCCEB, 0x5001E420, 0x24126EA1]


def test_rows_use_the_generator_as_described():
    seed, offset, start, H = 0x0123456789ABCDEF, 0xFEDCBA9876543210, (1 << 40) + 3, 24
    for p in (0.1, 0.5):
        keep, factor = ref.kept(2, H, p, seed, offset, start)
        assert factor == 65536 / (65536 - round(p * 65536))
        for t in range(2):
            for g in range(3):
                n = (start + t) * 3 + g
                words = ref.philox([n & 0xFFFFFFFF, n >> 32, offset & 0xFFFFFFFF, offset >> 32],
                                   [seed & 0xFFFFFFFF, seed >> 32])
                bits = [h for w in words for h in (w & 0xFFFF, w >> 16)]
                assert keep[t, 8 * g:8 * g + 8].tolist() == [b >= round(p * 65536) for b in bits]


@pytest.mark.parametrize("post", [False, True])
@pytest.mark.parametrize("gate", ["none", "channel", "token", "full"])
@pytest.mark.parametrize("p", [0.0, 0.3])
def test_norm_gradient(post, gate, p):
    g = torch.Generator().manual_seed(3)
    T, H = 5, 16
    rand = lambda *s: torch.randn(*s, dtype=torch.float64, generator=g).requires_grad_()  # noqa: E731
    h, y, w, wp = rand(T, H), rand(T, H), rand(H), rand(H) if post else None
    z = {"none": None, "channel": rand(H), "token": rand(T, 1), "full": rand(T, H)}[gate]
    dn, dh = rand(T, H).detach(), rand(T, H).detach()
    o = dict(weight=w, post_norm=post, post_weight=wp, gate=z, residual_scale=0.7, eps=1e-3, weight_offset=0.5, dropout=p,
             seed=7, offset=2)
    u, n, _, _ = ref.norm(h, y, **o)
    leaves = {"d_h": h, "d_y": y, "d_weight": w, "d_post_weight": wp, "d_gate": z}
    leaves = {k: v for k, v in leaves.items() if v is not None}
    auto = torch.autograd.grad((u * dh).sum() + (n * dn).sum(), list(leaves.values()))
    o = {k: v.detach() if isinstance(v, torch.Tensor) else v for k, v in o.items()}
    mine = ref.norm_backward(u.detach(), y.detach(), dn, dh, **o)
    for (k, leaf), a in zip(leaves.items(), auto):
        torch.testing.assert_close(mine[k][0], a, rtol=1e-12, atol=1e-13, msg=k)
        v = torch.randn(leaf.shape, dtype=torch.float64, generator=g)

        def value(step, leaf=leaf):
            moved = {id(leaf): leaf.detach() + step * v}
            at = lambda t: None if t is None else moved.get(id(t), t.detach())  # noqa: E731
            uu, nn, _, _ = ref.norm(at(h), at(y), **dict(o, weight=at(w), post_weight=at(wp), gate=at(z)))
            return float((uu * dh).sum() + (nn * dn).sum())

        # central differences: step^2 of the third derivative (about 1), rounding 1e-16 / step
        assert abs((value(1e-5) - value(-1e-5)) / 2e-5 - float((mine[k][0] * v).sum())) < 1e-7 * (1 + T * H)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("by_sequence", [False, True])
def test_balance_gradient(score, by_sequence):
    g = torch.Generator().manual_seed(5)
    T, E, K = 9, 6, 2
    l = torch.randn(T, E, dtype=torch.float64, generator=g)
    ids = torch.stack([torch.randperm(E, generator=g)[:K] for _ in range(T)])
    ids[2, 1] = -1
    mask = torch.tensor([1, 1, 0, 1, 1, 1, 1, 1, 0])
    cu = torch.tensor([0, 3, 3, 8, 9]) if by_sequence else None
    z = 0.1 if score == "softmax" else 0.0
    metrics, experts, counts, grad, _, _ = ref.balance(l, ids, 0.5, z, score, mask, cu)
    assert counts.tolist() == [7, 2 if by_sequence else 0] and int(experts.sum()) == 14
    v = torch.randn(T, E, dtype=torch.float64, generator=g)
    up, down = (float(ref.balance(l + s * v, ids, 0.5, z, score, mask, cu)[0][0]) for s in (1e-5, -1e-5))
    assert abs((up - down) / 2e-5 - float((grad * v).sum())) < 1e-8
    even = ref.balance(torch.zeros(4, 4), torch.arange(4)[:, None], 1.0)
    assert float(even[0][1]) == 1.0 and float(even[0][3]) == 1.0 and float(even[3].abs().max()) == 0.0
