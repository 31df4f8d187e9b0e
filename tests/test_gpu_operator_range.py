"""The trainer's attention and the serving weights at the ends of their ranges: gradients
of queries whose keys are few or whose weight is on few of them, more tokens than one
list of keys per tile, rollouts and pages past 2^32 bytes, views with a stride of 0,
calls side by side on two streams, padding behind the last token.

Tolerances.  A gradient is off, in 2-norm, by the roundings of p or ds and of the result:
each is at most half a step (2^-8 relative) and evenly spread over it (2^-8 / sqrt(3) of
the norm), and two of them are independent: 2^-8 sqrt(2/3).  Whatever of dq may be left
out for delta's sake is 0.001 of its norm.  Everything else is float32."""

import numpy as np
import pytest

from gpu_common import need_gpu, torch
from test_gpu_train import deaths, randn

pytestmark = pytest.mark.gpu

GRAD = 2.0 ** -8 * (2 / 3) ** 0.5 + 0.001


def exact(q, k, v, dout, death, scale, cap):
    """dq, dk, dv in 64 bits, on the GPU."""
    n, T, heads, _ = q.shape
    group = heads // k.shape[2]
    grads = [torch.zeros(x.shape, dtype=torch.float64, device="cuda") for x in (q, k, v)]
    t = torch.arange(T, device="cuda")
    for i in range(n):
        seen = (t[None] <= t[:, None]) & (t[:, None] < death[i][None])
        some = seen.any(1)
        for h in range(heads):
            g = h // group
            x, y, z, d = (a.double() for a in (q[i, :, h], k[i, :, g], v[i, :, g], dout[i, :, h]))
            s = x @ y.t().contiguous() * scale
            slope = torch.ones_like(s)
            if cap:
                th = torch.tanh(s / cap)
                s, slope = cap * th, 1 - th * th
            p = torch.softmax(s.masked_fill(~seen, -1e300), 1) * (seen & some[:, None])
            dp = d @ z.t().contiguous()
            ds = p * (dp - (p * dp).sum(1, keepdim=True)) * slope * scale
            grads[0][i, :, h] = ds @ y
            grads[1][i, :, g] += ds.t().contiguous() @ x
            grads[2][i, :, g] += p.t().contiguous() @ d
    return grads


def off(got, want):
    return float((got.double() - want).norm() / want.norm())


@pytest.mark.parametrize("T,H,G,dk,dv,doc,times,cap", [
    (257, 2, 2, 64, 64, 2, 1.0, 0.0), (390, 1, 3, 128, 128, 3, 1.0, 0.0), (300, 2, 1, 192, 128, 5, 1.0, 30.0),
    (513, 1, 2, 128, 128, 513, 16.0, 0.0), (500, 2, 1, 192, 128, 500, 16.0, 50.0), (260, 1, 1, 256, 256, 100, 8.0, 0.0),
    (700, 1, 2, 96, 96, 700, 1.0, 0.0)])
def test_gradients_where_a_weight_is_nearly_all(T, H, G, dk, dv, doc, times, cap):
    L = need_gpu()
    g = np.random.default_rng(T)
    kvs = L.KvsMask(0)
    q, k, v = randn(g, 1, T, H * G, dk) * times, randn(g, 1, T, H, dk), randn(g, 1, T, H, dv)
    dout = randn(g, 1, T, H * G, dv)
    t = np.arange(T)
    death = torch.from_numpy(np.minimum((t // doc + 1) * doc, T).astype(np.int32)[None]).cuda()
    out, lse = kvs.attend(q, k, v, death, cap=cap)
    got = kvs.attend_backward(dout, q, k, v, out, lse, death, cap=cap)
    for name, a, b in zip(("dq", "dk", "dv"), got, exact(q, k, v, dout, death, dk ** -0.5, cap)):
        assert off(a, b) <= GRAD, (name, off(a, b))
    kvs.close()


@pytest.mark.parametrize("T", [8193, 9000])
def test_epochs_longer_than_a_tile(T):
    L = need_gpu()
    g = np.random.default_rng(T)
    kvs = L.KvsMask(0)
    q, k, v, dout = randn(g, 1, T, 1, 64), randn(g, 1, T, 1, 64), randn(g, 1, T, 1, 64), randn(g, 1, T, 1, 64)
    death = np.full((1, T), T)
    for at in range(1000, T, 1000):   # half of what is left dies
        alive = np.flatnonzero((death[0] > at) & (np.arange(T) < at))
        death[0, g.permutation(alive)[:len(alive) // 2]] = at
    death = torch.from_numpy(death.astype(np.int32)).cuda()
    out, lse = kvs.attend(q, k, v, death)
    got = kvs.attend_backward(dout, q, k, v, out, lse, death)
    for name, a, b in zip(("dq", "dk", "dv"), got, exact(q, k, v, dout, death, 64 ** -0.5, 0.0)):
        assert off(a, b) <= GRAD, (name, off(a, b))
    kvs.close()


def test_rollouts_far_apart_in_memory():
    """Two rollouts more than 2^32 bytes apart, of which the kernels' tiles lie on both
    sides of that: bits as from one dense tensor."""
    L = need_gpu()
    g = np.random.default_rng(1)
    kvs = L.KvsMask(0)
    T, H, D, far = 131, 2, 64, (1 << 31) + 64
    room = torch.empty(far + 8 * T * H * D, dtype=torch.bfloat16, device="cuda")
    views = [room.as_strided((2, T, H, D), (far, H * D, D, 1), i * T * H * D) for i in range(8)]
    dense = [randn(g, 2, T, H, D) for _ in range(4)]
    for x, y in zip(views, dense):
        x.copy_(y)
    death = torch.from_numpy(deaths("cut", 2, T, g).astype(np.int32)).cuda()
    q, k, v, dout = dense
    out, lse = kvs.attend(q, k, v, death)
    want = (out, *kvs.attend_backward(dout, q, k, v, out, lse, death))
    q, k, v, dout, out, *grads = views
    _, lse = kvs.attend(q, k, v, death, out=out)
    kvs.attend_backward(dout, q, k, v, out, lse, death, grads=grads)
    for a, b in zip((out, *grads), want):
        assert torch.equal(a, b)
    kvs.close()


def test_strides_of_zero():
    """One value row for all tokens, one query for all heads, one rollout's keys for both:
    as the same values written out.  What is written may not overlap itself."""
    L = need_gpu()
    g = np.random.default_rng(2)
    kvs = L.KvsMask(0)
    n, T, H, D = 2, 70, 4, 64
    q = randn(g, n, T, 1, D).expand(n, T, H, D)
    k = randn(g, 1, T, H, D).expand(n, T, H, D)
    v = randn(g, n, 1, H, D).expand(n, T, H, D)
    dout = randn(g, n, T, 1, D).expand(n, T, H, D)
    death = torch.from_numpy(deaths("any", n, T, g).astype(np.int32)).cuda()
    out, lse = kvs.attend(q, k, v, death)
    got = (out, *kvs.attend_backward(dout, q, k, v, out, lse, death))
    q, k, v, dout = (x.contiguous() for x in (q, k, v, dout))
    out, lse = kvs.attend(q, k, v, death)
    for a, b in zip(got, (out, *kvs.attend_backward(dout, q, k, v, out, lse, death))):
        assert torch.equal(a, b)
    with pytest.raises(L.LeylineError):
        kvs.attend(q, k, v, death, out=out[:, :1].expand(n, T, H, D))
    kvs.close()


def test_two_calls_at_once():
    L = need_gpu()
    g = np.random.default_rng(3)
    kvs = L.KvsMask(0)
    sets = []
    for T, D in ((1100, 128), (700, 64)):
        x = [randn(g, 1, T, 4, D), randn(g, 1, T, 2, D), randn(g, 1, T, 2, D), randn(g, 1, T, 4, D)]
        sets.append((*x, torch.from_numpy(deaths("cut", 1, T, g).astype(np.int32)).cuda()))

    def both(q, k, v, dout, death, stream=None):
        out, lse = kvs.attend(q, k, v, death, cap=30.0, stream=stream)
        return (out, lse, *kvs.attend_backward(dout, q, k, v, out, lse, death, cap=30.0, stream=stream))

    want = [both(*s) for s in sets]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in sets]
    for _ in range(3):
        got = [both(*s, stream=t) for s, t in zip(sets, streams)]
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert all(torch.equal(x, y) for x, y in zip(a, b))
    kvs.close()


def test_padding_behind_the_last_token():
    """Keys of the padding die where they stand, and hold NaN: rows before them are as
    without the padding, rows of the padding are zeros with no weight, and no gradient."""
    L = need_gpu()
    g = np.random.default_rng(4)
    kvs = L.KvsMask(0)
    T, pad, H, D = 190, 70, 2, 128
    q, k, v, dout = (randn(g, 1, T + pad, H, D) for _ in range(4))
    for x in (k, v):
        x[:, T:] = float("nan")
    death = torch.full((1, T + pad), T, dtype=torch.int32, device="cuda")
    death[0, T:] = torch.arange(T, T + pad)
    out, lse = kvs.attend(q, k, v, death)
    dq, dk, dv = kvs.attend_backward(dout, q, k, v, out, lse, death)
    assert torch.isinf(lse[:, T:]).all()
    for x in (out, dq, dk, dv):
        assert (x[:, T:] == 0).all() and torch.isfinite(x).all()
    short = [x[:, :T].contiguous() for x in (q, k, v, dout)]
    o, l = kvs.attend(*short[:3], death[:, :T].contiguous())
    for a, b in zip((out, dq, dk, dv), (o, *kvs.attend_backward(short[3], *short[:3], o, l, death[:, :T].contiguous()))):
        assert off(a[:, :T], b.double()) <= 2 * GRAD
    kvs.close()


@pytest.mark.parametrize("gqa", [False, True])
def test_pages_past_32_bits(gqa):
    """A sequence whose pages lie on both sides of 2^32 bytes of a layer: the weights are
    those of the same rows in a small pool."""
    L = need_gpu()
    g = np.random.default_rng(5)
    P, n, heads = 64, 300, 8
    row = (2, 128) if gqa else (576,)
    width = int(np.prod(row))
    far = (1 << 32) // (2 * width * P)   # the page that 2^32 bytes lie in
    q = randn(g, 3, heads, 128 if gqa else 576)
    rows = [randn(g, n, *row) for _ in range(2 if gqa else 1)]
    results = []
    for pages, order in ((8, [5, 0, 3, 1, 6]), (far + 8, [far + 5, 0, far, far - 1, far + 1])):
        planes = [torch.empty((1, pages, P, *row), dtype=torch.bfloat16, device="cuda") for _ in rows]
        for x, y in zip(planes, rows):
            for i, page in enumerate(order):
                part = y[i * P:(i + 1) * P]
                x[0, page, :len(part)] = part
        table = torch.full((1, 6), -1, dtype=torch.int32, device="cuda")
        pool = L.GqaPool(*planes, table, rotary_dim=64) if gqa else L.Pool(planes[0], table)
        pool.seq_set_pages(0, order, n)
        step = pool.step(heads, max_tokens=3)
        step.begin([0], [3], grow=False)
        out, lse = step.attend(0, q, scale=0.1, lse=True, cap=20.0)
        w = torch.zeros((1, 6 * P), device="cuda")
        step.weigh(0, q, lse, w, scale=0.1, cap=20.0)
        torch.cuda.synchronize()
        results.append((out, lse, w[:, :n].clone()))
        step.close()
        pool.close()
    for a, b in zip(*results):
        assert torch.equal(a, b)


@pytest.mark.parametrize("n,T,H,G,dk,dv,cap", [(2, 150, 1, 1, 136, 192, 0.0), (1, 140, 2, 2, 8, 256, 0.0), (1, 133, 1, 2, 256, 8, 20.0),
                                               (1, 200, 1, 3, 200, 64, 0.0), (400, 5, 1, 1, 64, 64, 0.0), (1, 70, 1, 64, 64, 64, 0.0),
                                               (1, 1000, 1, 1, 72, 40, 10.0)])
def test_odd_widths_and_counts(n, T, H, G, dk, dv, cap):
    L = need_gpu()
    g = np.random.default_rng(n + T + dk)
    kvs = L.KvsMask(0)
    q, k, v, dout = randn(g, n, T, H * G, dk), randn(g, n, T, H, dk), randn(g, n, T, H, dv), randn(g, n, T, H * G, dv)
    death = torch.from_numpy(deaths("cut", n, T, g).astype(np.int32)).cuda()
    out, lse = kvs.attend(q, k, v, death, cap=cap)
    got = kvs.attend_backward(dout, q, k, v, out, lse, death, cap=cap)
    for name, a, b in zip(("dq", "dk", "dv"), got, exact(q, k, v, dout, death, dk ** -0.5, cap)):
        assert off(a, b) <= GRAD, (name, off(a, b))
    kvs.close()


def test_no_rollouts():
    L = need_gpu()
    kvs = L.KvsMask(0)
    q, k, v = (torch.empty((0, 9, h, 64), dtype=torch.bfloat16, device="cuda", requires_grad=True) for h in (4, 2, 2))
    death = torch.empty((0, 9), dtype=torch.int32, device="cuda")
    out = kvs.attention(q, k, v, death)
    out.sum().backward()
    assert out.shape == (0, 9, 4, 64) and q.grad.shape == q.shape and v.grad.shape == v.shape
    with pytest.raises((ValueError, L.LeylineError)):
        kvs.attend(q[:, :0], k[:, :0], v[:, :0], death[:, :0])
    with pytest.raises((ValueError, L.LeylineError)):
        kvs.attend(q, k, v, death.long())
    kvs.close()


def test_weights_in_wider_rows_and_a_budget_of_nothing():
    """A selection over weights whose rows lie apart in a wider tensor; a budget of no rows
    keeps none, one past the rows keeps all, and other sequences' weights stay."""
    L = need_gpu()
    table = torch.full((3, 20), -1, dtype=torch.int32, device="cuda")
    pool = L.Pool(torch.zeros((1, 64, 16, 576), dtype=torch.bfloat16, device="cuda"), table)
    lens = [0, 100, 300]
    seqs = [pool.seq_alloc(n) for n in lens]
    wide = torch.rand((3, 1000), device="cuda")
    before = wide.clone()
    keep, offsets = pool.keep_heaviest(seqs[1:], [0, 400], wide, kept_weights=wide)
    torch.cuda.synchronize()
    assert not keep[:100].any() and keep[100:400].all() and list(offsets) == [0, 100]
    before[seqs[1], :100] = 0   # (zeros up to the old length)
    assert torch.equal(wide, before)
    keep, _ = pool.keep_heaviest([seqs[2]], [7], wide, sinks=2, recent=2, kept_weights=wide)
    torch.cuda.synchronize()
    kept = torch.nonzero(keep[:300]).flatten()
    assert len(kept) == 7 and kept[:2].tolist() == [0, 1] and kept[-2:].tolist() == [298, 299]
    assert torch.equal(wide[seqs[2], :7], before[seqs[2]][kept]) and torch.equal(wide[seqs[1]], before[seqs[1]])
    assert torch.equal(wide[:, 300:], before[:, 300:])
    pool.close()
