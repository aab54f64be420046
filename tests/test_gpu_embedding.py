"""lp_embedding and lp_embedding_backward on the GPU against the fp64 oracle.

The lookup is compared bit for bit with the fp32 product. The gradient of an id with n positions is
a sum of n fp32 values in some order, then one product: each element may be off by (n + 1) 2^-24 of
the sum of the magnitudes (and half a bf16 step where it is stored in bf16)."""
import numpy as np
import pytest

from lp_util import dev_i32
from oracle import train

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


def _part(lp, real, bounds, local=False):
    return lp.VocabPartition(real, bounds[-1] if not local else max(bounds[-1], real),
                             tuple((bounds[i], bounds[i + 1]) for i in range(len(bounds) - 1)), local=local)


def _rand(shape, dtype, seed):
    import torch
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return torch.empty(shape, dtype=dtype, device="cuda").normal_(generator=g)


def _dtype(name):
    import torch
    return {"bf16": torch.bfloat16, "f32": torch.float32}[name]


PARTS = [(1000, [0, 1000]), (997, [0, 200, 200, 600, 1024]), (513, [0, 8, 16, 500, 501, 513, 513, 513, 513])]


@pytest.mark.parametrize("table", ["bf16", "f32"])
@pytest.mark.parametrize("out", ["bf16", "f32"])
@pytest.mark.parametrize("T,H,part", [(1, 8, 0), (3, 264, 1), (257, 1032, 2), (64, 4096, 0), (1000, 72, 1)])
def test_lookup(lp, table, out, T, H, part):
    import torch
    real, bounds = PARTS[part]
    rs = np.random.RandomState(T + H)
    ids = rs.randint(-1, real, T)
    ids[0] = real - 1
    W = [_rand((b - a, H), _dtype(table), 7 + a) if b > a else None for a, b in zip(bounds[:-1], bounds[1:])]
    for scale in (1.0, 0.37, -64.0):
        y = lp.lp_embedding(dev_i32(ids), W, _part(lp, real, bounds), scale=scale, out_dtype=_dtype(out))
        full = torch.cat([w for w in W if w is not None]).float()
        at = torch.from_numpy(np.maximum(ids, 0)).cuda()
        want = torch.where(torch.from_numpy(ids >= 0).cuda()[:, None],
                           full[at] * torch.tensor(scale, dtype=torch.float32, device="cuda"), 0.0).to(_dtype(out))
        assert torch.equal(y, want)
        oracle = train.embedding(ids, full.double().cpu().numpy(), 0, float(np.float32(scale)))
        # half an ulp of the output type, and of fp32 before it
        half = (2.0 ** -8 if out == "bf16" else 2.0 ** -24) + 2.0 ** -24
        assert np.all(np.abs(y.double().cpu().numpy() - oracle) <= np.abs(oracle) * half * 1.001 + 1e-38)
    assert lp.lp_get_device_error() == 0


@pytest.mark.parametrize("H", [8, 16, 24, 32, 40, 64, 120, 128, 136])
@pytest.mark.parametrize("T", [1, 3, 127, 1000, 100003, 1250007])
def test_lookup_of_few_columns(lp, H, T):
    import torch
    V = 5000
    W = _rand((V, H), torch.bfloat16, H)
    ids = np.random.RandomState(T).randint(-1, V, T)
    i = dev_i32(ids)
    buf = torch.full((T + 2, H), 3.0, device="cuda")
    y = lp.lp_embedding(i, [W], _part(lp, V, [0, V]), scale=1.5, out=buf[1:T + 1])
    want = torch.where((i >= 0)[:, None], W[i.long().clamp(min=0)].float() * 1.5, 0.0)
    assert torch.equal(y, want) and bool((buf[0] == 3).all()) and bool((buf[T + 1] == 3).all())
    assert lp.lp_get_device_error() == 0


def test_lookup_rank_local_strided_and_refused_ids(lp):
    import torch
    real, H = 1000, 136
    full = _rand((real, H), torch.bfloat16, 1)
    ids = dev_i32(np.array([0, 399, 400, 699, 700, 999, -1]))
    lo = lp.lp_embedding(ids, [full[:400].contiguous()], _part(lp, real, [0, 400], local=True))
    mid = lp.lp_embedding(ids, [full[400:700].contiguous()], _part(lp, real, [400, 700], local=True))
    hi = lp.lp_embedding(ids, [full[700:].contiguous()], _part(lp, real, [700, 1000], local=True))
    whole = lp.lp_embedding(ids, [full], _part(lp, real, [0, 1000]))
    assert torch.equal(lo + mid + hi, whole) and torch.count_nonzero(lo[2:]) == 0
    assert lp.lp_get_device_error() == 0
    # a view with a longer row stride; what lies between the rows is left alone
    buf = torch.full((7, H + 24), 5.0, dtype=torch.bfloat16, device="cuda")
    lp.lp_embedding(ids, [full], _part(lp, real, [0, 1000]), out=buf[:, 8:8 + H])
    assert torch.equal(buf[:, 8:8 + H], whole)
    assert bool((buf[:, :8] == 5).all()) and bool((buf[:, 8 + H:] == 5).all())
    for bad in (1000, -2, 2 ** 31 - 1, -2 ** 31):
        y = lp.lp_embedding(dev_i32(np.array([5, bad])), [full], _part(lp, real, [0, 1000]))
        assert torch.equal(y[0], full[5]) and torch.count_nonzero(y[1]) == 0
        assert lp.lp_get_device_error() == 11
    # NaN and infinities of the table come through
    full[3, 0], full[3, 1] = float("nan"), float("inf")
    y = lp.lp_embedding(dev_i32([3]), [full], _part(lp, real, [0, 1000]), scale=2.0)
    assert bool(y[0, 0].isnan()) and bool(y[0, 1].isinf())
    assert lp.lp_embedding(dev_i32(np.zeros(0)), [full], _part(lp, real, [0, 1000])).shape == (0, H)
    assert lp.lp_get_device_error() == 0


def _ids(kind, T, real, rs):
    ids = np.minimum((real ** rs.rand(T)).astype(np.int64) - 1, real - 1)
    if kind == "hot":
        ids[rs.rand(T) < 0.8] = real // 2
    elif kind == "one":
        ids[:] = real - 1
    elif kind == "distinct":
        ids = rs.permutation(max(real, T))[:T] % real
    elif kind == "unused":
        ids[:] = -1
    elif kind == "runs":                              # lengths around the 32-position chunk, and far above
        ids = np.repeat(np.arange(real), np.resize([1, 31, 32, 33, 64, 65, 2, 30, 97, 5], real))[:T]
        ids = rs.permutation(np.resize(ids, T))
    ids[rs.rand(T) < 0.1] = -1
    return ids


def _check_gradient(got, bf16, want, mag, n):
    got = got.double().cpu().numpy()
    bound = (n[:, None] + 1) * 2.0 ** -24 * mag * 1.01
    if bf16:
        bound = bound + (np.abs(want) + bound) * 2.0 ** -8
    assert np.all(np.abs(got - want) <= bound + 1e-38)
    assert np.all(got[n == 0] == 0)


@pytest.mark.parametrize("grad,dw", [("bf16", "f32"), ("f32", "f32"), ("bf16", "bf16"), ("f32", "bf16")])
@pytest.mark.parametrize("kind", ["zipf", "hot", "one", "distinct", "unused", "runs"])
@pytest.mark.parametrize("T,H,part", [(1, 8, 0), (31, 264, 1), (33, 256, 2), (1000, 136, 1), (4099, 72, 0)])
def test_gradient(lp, grad, dw, kind, T, H, part):
    import torch
    real, bounds = PARTS[part]
    rs = np.random.RandomState(T * 7 + H)
    ids = _ids(kind, T, real, rs)
    dY = _rand((T, H), _dtype(grad), 3)
    out = lp.lp_embedding_backward(dev_i32(ids), dY, _part(lp, real, bounds), scale=0.75, dw_dtype=_dtype(dw))
    host = dY.double().cpu().numpy()
    want, mag, n = train.embedding_backward(ids, host, 0, bounds[-1], 0.75)
    got = torch.cat([g for g in out if g is not None])
    _check_gradient(got, dw == "bf16", want, mag, n)
    again = lp.lp_embedding_backward(dev_i32(ids), dY, _part(lp, real, bounds), scale=0.75, dw_dtype=_dtype(dw))
    assert all(a is None or torch.equal(a, b) for a, b in zip(out, again))
    assert lp.lp_get_device_error() == 0


@pytest.mark.parametrize("kind", ["zipf", "hot", "one", "runs", "unused"])
@pytest.mark.parametrize("T", [32, 63, 64, 65, 96, 127, 128, 129, 257, 513, 1024, 1025, 1535, 1536, 1537, 2049])
@pytest.mark.parametrize("acc", [False, True])
def test_gradient_where_the_method_changes(lp, kind, T, acc):
    """Around the batches from which runs are cut, and from which positions are sorted by digits."""
    import torch
    real, bounds, H = 997, [0, 200, 200, 600, 1024], 264
    rs = np.random.RandomState(T)
    ids = _ids(kind, T, real, rs)
    dY = _rand((T, H), torch.float32, T + 1)
    part, i = _part(lp, real, bounds), dev_i32(ids)
    want, mag, n = train.embedding_backward(ids, dY.double().cpu().numpy(), 0, bounds[-1], 0.75)
    fresh = lp.lp_embedding_backward(i, dY, part, scale=0.75,
                                     dW=[torch.full((b - a, H), 7.0, device="cuda") for a, b in zip(bounds[:-1], bounds[1:])])
    _check_gradient(torch.cat(fresh), False, want, mag, n)
    if acc:
        base = [_rand((b - a, H), torch.float32, a) for a, b in zip(bounds[:-1], bounds[1:])]
        dW = [b.clone() for b in base]
        lp.lp_embedding_backward(i, dY, part, scale=0.75, accumulate=True, dW=dW)
        assert all(torch.equal(d, b + f) for d, b, f in zip(dW, base, fresh))
    else:
        again = lp.lp_embedding_backward(i, dY, part, scale=0.75)
        assert all(torch.equal(x, y) for x, y in zip(again, fresh) if x is not None)
    assert lp.lp_get_device_error() == 0


@pytest.mark.parametrize("T,H,grad,dw,kind", [(20011, 16, "bf16", "f32", "zipf"), (70001, 8, "f32", "bf16", "hot"),
                                              (16384, 264, "bf16", "f32", "runs"), (5000, 40, "bf16", "bf16", "zipf"),
                                              (100003, 8, "bf16", "f32", "zipf")])
def test_gradient_of_long_batches(lp, T, H, grad, dw, kind):
    """Sorted by clusters of 8 and 16 CTAs, in two and three digits, with the positions kept in registers
    and not; long runs joined from many pieces."""
    import torch
    for real, bounds in ((1000, [0, 1000]), (300000, [0, 100000, 100000, 300032])):
        ids = _ids(kind, T, real, np.random.RandomState(T))
        dY = _rand((T, H), _dtype(grad), 6)
        out = lp.lp_embedding_backward(dev_i32(ids), dY, _part(lp, real, bounds), scale=2.0, dw_dtype=_dtype(dw))
        want, mag, n = train.embedding_backward(ids, dY.double().cpu().numpy(), 0, bounds[-1], 2.0)
        _check_gradient(torch.cat([g for g in out if g is not None]), dw == "bf16", want, mag, n)
    assert lp.lp_get_device_error() == 0


@pytest.mark.parametrize("kind", ["spread", "dense"])
@pytest.mark.parametrize("T", [1, 60, 600, 1537, 2000, 20000, 40000, 98304, 100000])
def test_gradient_of_large_tables(lp, kind, T):
    """A table of 300 MB, most of whose rows get zeros according to the marks of the named ones, over every method
    of sorting. Whole numbers, so that every order of summation gives the same."""
    import torch
    V, H = 1200000, 64
    rs = np.random.RandomState(T)
    ids = rs.randint(-1, V, T) if kind == "spread" else V - 1 - rs.randint(0, 3 * T, T)
    ids[rs.rand(T) < 0.05] = V - 3
    dY = torch.from_numpy(rs.randint(-8, 9, (T, H)).astype(np.float32)).cuda()
    dW = [torch.full((500000, H), 7.0, device="cuda"), torch.full((V - 500000, H), 7.0, device="cuda")]
    i = dev_i32(ids)
    lp.lp_embedding_backward(i, dY, _part(lp, V, [0, 500000, V]), scale=2.0, dW=dW)
    used = (i >= 0)[:, None]
    want = torch.zeros((V, H), device="cuda").index_add_(0, i.long().clamp(min=0), torch.where(used, dY * 2, 0.0))
    assert torch.equal(torch.cat(dW), want)
    assert lp.lp_get_device_error() == 0


@pytest.mark.parametrize("kind", ["zipf", "hot", "runs"])
def test_gradient_accumulates_one_add_per_element(lp, kind):
    import torch
    real, bounds = PARTS[1]
    T, H = 3001, 136
    ids = _ids(kind, T, real, np.random.RandomState(9))
    dY = _rand((T, H), torch.bfloat16, 5)
    part = _part(lp, real, bounds)
    fresh = lp.lp_embedding_backward(dev_i32(ids), dY, part, scale=3.0)
    held = [_rand((b - a, H), torch.float32, 11 + a) if b > a else None for a, b in zip(bounds[:-1], bounds[1:])]
    before = [None if h is None else h.clone() for h in held]
    lp.lp_embedding_backward(dev_i32(ids), dY, part, scale=3.0, accumulate=True, dW=held)
    for h, b, f in zip(held, before, fresh):
        assert h is None or torch.equal(h, b + f)
    # an empty batch: zeros, or nothing when accumulating
    none, dY0 = dev_i32(np.zeros(0)), torch.empty((0, H), dtype=torch.bfloat16, device="cuda")
    lp.lp_embedding_backward(none, dY0, part, accumulate=True, dW=held)
    assert all(h is None or torch.equal(h, b + f) for h, b, f in zip(held, before, fresh))
    assert all(z is None or torch.count_nonzero(z) == 0 for z in lp.lp_embedding_backward(none, dY0, part, dW=held))


def test_gradient_rank_local_strided_and_refused_ids(lp):
    import torch
    real, T, H = 1000, 777, 200
    rs = np.random.RandomState(2)
    ids = _ids("hot", T, real, rs)
    buf = _rand((T, H + 40), torch.bfloat16, 4)
    dY = buf[:, 16:16 + H]
    whole = lp.lp_embedding_backward(dev_i32(ids), dY, _part(lp, real, [0, 400, 1000]))
    want, mag, n = train.embedding_backward(ids, dY.double().cpu().numpy(), 0, real, 1.0)
    _check_gradient(torch.cat(whole), False, want, mag, n)
    a = lp.lp_embedding_backward(dev_i32(ids), dY, _part(lp, real, [0, 400], local=True))
    b = lp.lp_embedding_backward(dev_i32(ids), dY, _part(lp, real, [400, 1000], local=True))
    for got, lo, hi in ((a[0], 0, 400), (b[0], 400, 1000)):
        _check_gradient(got, False, want[lo:hi], mag[lo:hi], n[lo:hi])
    assert lp.lp_get_device_error() == 0
    # a refused id takes no part; a NaN stays in its own row, and an unused position's is never read
    bad = ids.copy()
    bad[5], bad[6] = real, -7
    got = lp.lp_embedding_backward(dev_i32(bad), dY, _part(lp, real, [0, 400, 1000]))
    assert lp.lp_get_device_error() == 11
    want, mag, n = train.embedding_backward(np.where((bad < 0) | (bad >= real), -1, bad), dY.double().cpu().numpy(), 0,
                                            real, 1.0)
    _check_gradient(torch.cat(got), False, want, mag, n)
    ids[:] = np.arange(T)
    ids[10] = -1
    nan = dY.contiguous()
    nan[10], nan[11] = float("nan"), float("nan")
    got = torch.cat(lp.lp_embedding_backward(dev_i32(ids), nan, _part(lp, real, [0, 400, 1000])))
    assert bool(got[11].isnan().all()) and int(got.isnan().any(dim=1).sum()) == 1
    assert lp.lp_get_device_error() == 0


def test_offsets_past_32_bits(lp):
    """Tables and batches of more than 2^31 elements: the rows at their far ends."""
    import torch
    V, H = 530001, 4096
    part = _part(lp, V, [0, V])
    W = torch.zeros((V, H), dtype=torch.bfloat16, device="cuda")
    W[V - 1], W[V - 2], W[0] = 3.0, 2.0, 1.0
    y = lp.lp_embedding(dev_i32([V - 1, 0, V - 2, 5]), [W], part)
    assert y.float().mean(dim=1).tolist() == [3.0, 1.0, 2.0, 0.0]
    # a batch as large: the table of a few rows, the named positions at both ends
    small = _part(lp, 40, [0, 40])
    ids = np.full(V, -1)
    ids[[0, V - 1]], ids[V - 2], ids[V - 40:V - 2] = 39, 7, 38
    dY = W                                          # row V-1 threes, row V-2 twos, row 0 ones
    g = lp.lp_embedding_backward(dev_i32(ids), dY, small)[0]
    want = torch.zeros(40, device="cuda")
    want[39], want[7] = 4.0, 2.0
    assert torch.equal(g, want[:, None].expand(40, H))
    y = lp.lp_embedding(dev_i32(ids), [W[:40].contiguous()], small)
    assert int(torch.count_nonzero(y)) == 0 and y.shape == (V, H)
    # a gradient as large
    ones = torch.ones((5, H), dtype=torch.bfloat16, device="cuda")
    g = lp.lp_embedding_backward(dev_i32([V - 1, 0, V - 1, -1, V - 2]), ones, part, dw_dtype=torch.bfloat16)[0]
    sums = g.sum(dim=1, dtype=torch.float32)
    assert sums[[V - 1, V - 2, 0]].tolist() == [2.0 * H, 1.0 * H, 1.0 * H]
    assert float(sums.sum()) == 4.0 * H
    assert lp.lp_get_device_error() == 0


def test_gradient_is_the_transpose_of_the_lookup(lp):
    """<lookup(V), dY> = <V, gradient(dY)> for any V: on integers, where fp32 is exact."""
    import torch
    real, T, H = 300, 2000, 64
    rs = np.random.RandomState(8)
    ids = dev_i32(_ids("hot", T, real, rs))
    V = torch.from_numpy(rs.randint(-3, 4, (real, H)).astype(np.float32)).cuda()
    dY = torch.from_numpy(rs.randint(-3, 4, (T, H)).astype(np.float32)).cuda()
    part = _part(lp, real, [0, real])
    y = lp.lp_embedding(ids, [V], part, scale=2.0)
    g = lp.lp_embedding_backward(ids, dY, part, scale=2.0)[0]
    assert float((y.double() * dY.double()).sum()) == float((V.double() * g.double()).sum())


def test_streams_and_graph(lp):
    """The calls run on the caller's stream and can be captured."""
    import torch
    real, T, H = 500, 600, 128
    part = _part(lp, real, [0, real])
    ids = dev_i32(_ids("hot", T, real, np.random.RandomState(3)))
    W, dY = _rand((real, H), torch.bfloat16, 1), _rand((T, H), torch.bfloat16, 2)
    y0, g0 = lp.lp_embedding(ids, [W], part), lp.lp_embedding_backward(ids, dY, part)[0]
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        y1, g1 = lp.lp_embedding(ids, [W], part), lp.lp_embedding_backward(ids, dY, part)[0]
    s.synchronize()
    assert torch.equal(y0, y1) and torch.equal(g0, g1)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y2, g2 = lp.lp_embedding(ids, [W], part), lp.lp_embedding_backward(ids, dY, part)[0]
    for _ in range(3):
        y2.zero_()
        g2.fill_(7.0)
        graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(y0, y2) and torch.equal(g0, g2)
