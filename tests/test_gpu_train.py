"""GPU parity of the trainer's attention and its gradients (include/leyline_train.h)
against the float64 oracle, through the binding: head layouts and widths, lengths
from one token, death times of every kind, views, what is not seen holding NaN.

Tolerances.  A product of d values summed in float32 is off by at most d 2^-24 of the
sum of magnitudes; a score's error shifts its weight by that relatively, and so do the
roundings of the exponent (2^-24 of score and lse, a few times: 8 2^-24 (1 + |s| + |lse|))
and of the tanh (2^-21 of the score).  Weights and the scores' gradients are rounded to
bf16 for the products (half a step, 2^-8), results once more.  delta is a sum over the
rounded out, which is off by 2^-8 (|out| + sum p |v|) and more.  Float32 sums over n
terms add n 2^-24 of the magnitudes."""

import numpy as np
import pytest

from oracle import weight_oracle as W

from gpu_common import need_gpu, torch

pytestmark = pytest.mark.gpu

H = 2.0 ** -8
F = 2.0 ** -24


def f64(t):
    return t.detach().float().cpu().numpy().astype(np.float64)


def randn(g, *shape):
    return torch.from_numpy(g.standard_normal(shape).astype(np.float32)).to(torch.bfloat16).cuda()


def deaths(kind, n, T, g):
    t = np.arange(T)
    if kind == "all":
        return np.full((n, T), T)
    if kind == "doc":
        return np.stack([np.minimum((t // (d := 3 + 17 * i) + 1) * d, T) for i in range(n)])
    if kind == "any":      # whatever an int32 may hold
        d = g.integers(-3, 2 * T + 2, (n, T))
        d[g.random((n, T)) < 0.1] = 2 ** 31 - 1
        d[g.random((n, T)) < 0.05] = -2 ** 31
        return d
    assert kind == "cut"   # an engine's evictions, and padding
    out = np.full((n, T), T)
    for i in range(n):
        length = max(1, T - 5 * i)
        for at in range(max(1, T // 4), length, max(1, T // 3)):
            alive = np.flatnonzero((out[i] > at) & (t < at))
            out[i, g.permutation(alive)[:len(alive) // 2]] = at
        out[i, length:] = t[length:]
    return out


def check(q, k, v, dout, death, scale, cap, out, lse, grads, what=("out", "dq", "dk", "dv")):
    """Every value against the oracle; prints the worst error over its tolerance."""
    n, T, heads, dk = q.shape
    group = heads // k.shape[2]
    gq, gk, gv = (np.zeros(x.shape) for x in (q, k, v))
    tq, tk, tv = (np.zeros(x.shape) for x in (q, k, v))
    worst = {}
    fq, fk, fv, fo, fl, fd = (f64(x) if x is not None else None for x in (q, k, v, out, lse, dout))

    def near(name, got, want, tol):
        assert np.array_equal(np.isfinite(got), np.isfinite(want)), name
        fine = np.isfinite(want)
        e = np.abs(np.where(fine, got, 0.0) - np.where(fine, want, 0.0)) / (tol + 1e-30)
        worst[name] = max(worst.get(name, 0.0), float(e.max(initial=0.0)))
        assert worst[name] <= 1, (name, worst[name], np.argwhere(e > 1)[:4].tolist())

    for i in range(n):
        seen = W.death_seen(death[i])
        for h in range(heads):
            g = h // group
            x, y, z = fq[i, :, h], fk[i, :, g], fv[i, :, g]
            # what is not seen does not count, and NaN there must not reach the oracle either
            y, z = np.where(seen.any(0)[:, None], y, 0.0), np.where(seen.any(0)[:, None], z, 0.0)
            xs = np.where(seen.any(1)[:, None], x, 0.0)
            raw = scale * (xs @ y.T)
            sc = W.capped(raw, cap)
            p, lo = W.softmax(sc, seen)
            slack = abs(scale) * (np.abs(xs) @ np.abs(y).T)
            ll = np.where(np.isfinite(lo), lo, 0.0)[:, None]
            # a weight's relative error
            ew = np.where(seen, dk * F * slack + 8 * F * (1 + np.abs(sc) + np.abs(ll)) + (2.0 ** -21 * np.abs(sc) if cap else 0), 0)
            top = ew.max(1, initial=0.0)[:, None]
            o = p @ z
            mag = p @ np.abs(z)
            near("lse", fl[i, :, h], lo, top[:, 0] + T * F + 4 * F * np.abs(ll[:, 0]))
            eo = H * (np.abs(o) + mag) + (2 * top + 2 * T * F) * mag
            near("out", fo[i, :, h], o, eo)
            if grads is None:
                continue
            do = np.where(seen.any(1)[:, None], fd[i, :, h], 0.0)
            dp, ado = do @ z.T, np.abs(do)
            delta = (do * o).sum(-1, keepdims=True)
            slope = 1 - np.tanh(raw / cap) ** 2 if cap else np.ones_like(raw)
            ds = p * (dp - delta) * scale * slope
            rel = ew + top + T * F + 2 * F
            eds = np.abs(ds) * (H + rel + 8 * F) + p * abs(scale) * (
                slope * (z.shape[1] * F * (ado @ np.abs(z).T) + (ado * eo).sum(-1, keepdims=True)
                         + z.shape[1] * F * (ado * (np.abs(o) + eo)).sum(-1, keepdims=True))
                + (2.0 ** -20 * np.abs(dp - delta) if cap else 0) + (2 * dk * F * slack / cap * np.abs(dp - delta) if cap else 0))
            gq[i, :, h] = ds @ y
            gk[i, :, g] += ds.T @ xs
            gv[i, :, g] += p.T @ do
            tq[i, :, h] = eds @ np.abs(y) + T * F * (np.abs(ds) @ np.abs(y))
            tk[i, :, g] += eds.T @ np.abs(xs) + group * T * F * (np.abs(ds).T @ np.abs(xs))
            tv[i, :, g] += (p * (H + rel + group * T * F)).T @ ado
    if grads is not None:
        for name, got, want, tol in (("dq", grads[0], gq, tq), ("dk", grads[1], gk, tk), ("dv", grads[2], gv, tv)):
            near(name, f64(got), want, H * np.abs(want) + tol)
    print(" ".join(f"{a} {b:.2f}" for a, b in worst.items()), flush=True)


def run(n, T, kv_heads, group, dk, dv, kind, cap=0.0, scale=None, seed=0, times=1.0):
    L = need_gpu()
    g = np.random.default_rng(seed)
    kvs = L.KvsMask(0)
    q, k, v = randn(g, n, T, kv_heads * group, dk) * times, randn(g, n, T, kv_heads, dk), randn(g, n, T, kv_heads, dv)
    dout = randn(g, n, T, kv_heads * group, dv)
    death = deaths(kind, n, T, g)
    d = torch.from_numpy(death.astype(np.int32)).cuda()
    s = dk ** -0.5 if scale is None else scale
    out, lse = kvs.attend(q, k, v, d, scale=scale, cap=cap)
    grads = kvs.attend_backward(dout, q, k, v, out, lse, d, scale=scale, cap=cap)
    torch.cuda.synchronize()
    check(q, k, v, dout, death, s, cap, out, lse, grads)
    kvs.close()


SHAPES = [
    # n, tokens, KV heads, group, key width, value width, mask
    (1, 1, 1, 1, 8, 8, "all"),
    (2, 2, 1, 3, 64, 64, "any"),
    (1, 31, 2, 1, 32, 32, "all"),
    (1, 64, 1, 2, 128, 128, "all"),
    (1, 65, 2, 2, 128, 128, "cut"),
    (2, 63, 1, 1, 64, 64, "doc"),
    (3, 127, 1, 2, 96, 96, "cut"),
    (1, 129, 3, 1, 80, 80, "doc"),
    (1, 257, 2, 4, 128, 128, "cut"),
    (2, 200, 2, 1, 192, 128, "cut"),
    (1, 389, 1, 2, 192, 128, "all"),
    (1, 150, 1, 2, 256, 256, "cut"),
    (1, 333, 1, 1, 128, 64, "any"),
    (1, 190, 2, 1, 64, 128, "cut"),
    (2, 100, 1, 1, 8, 200, "any"),
    (1, 100, 1, 1, 200, 8, "doc"),
    (1, 700, 1, 5, 64, 64, "cut"),
    (1, 513, 1, 1, 128, 128, "doc"),
    (1, 40, 12, 1, 16, 24, "any"),
]


@pytest.mark.parametrize("n,T,kv_heads,group,dk,dv,kind", SHAPES)
@pytest.mark.parametrize("cap", [0.0, 5.0])
def test_matches_the_oracle(n, T, kv_heads, group, dk, dv, kind, cap):
    run(n, T, kv_heads, group, dk, dv, kind, cap, seed=T)


@pytest.mark.parametrize("scale,cap,times", [(-0.3, 0.0, 1.0), (0.0, 0.0, 1.0), (0.0, 30.0, 1.0), (-1.0, 2.0, 1.0),
                                              (0.7, 50.0, 4.0), (3.0, 0.0, 8.0), (0.05, 1e-3, 1.0), (0.1, 1e6, 1.0)])
def test_scales_and_caps(scale, cap, times):
    run(1, 140, 1, 2, 64, 64, "cut", cap, scale, seed=7, times=times)


@pytest.mark.parametrize("kind", ["cut", "doc", "any"])
@pytest.mark.parametrize("dk,dv", [(64, 64), (128, 128), (192, 128), (256, 256)])
def test_what_is_not_seen_may_hold_anything(kind, dk, dv):
    """Keys that nobody sees hold NaN and infinities, and queries that see nothing;
    then one key and one query that some see: only those get NaN."""
    L = need_gpu()
    g = np.random.default_rng(3)
    n, T, Hk, G = 2, 210, 2, 2
    kvs = L.KvsMask(0)
    q, k, v = randn(g, n, T, Hk * G, dk), randn(g, n, T, Hk, dk), randn(g, n, T, Hk, dv)
    dout = randn(g, n, T, Hk * G, dv)
    death = deaths(kind, n, T, g)
    death[:, 50:60] = np.arange(50, 60)      # nobody sees these
    death[:, 130] = 0
    death[1, :33] = 20                       # and these queries see nothing
    death[1, 20:33] = np.arange(20, 33)
    at, head = 70, 1
    death[0, at], death[0, 120] = 100, T
    for i in range(n):
        seen = W.death_seen(death[i])
        gone = torch.from_numpy(np.flatnonzero(~seen.any(0))).cuda()
        blind = torch.from_numpy(np.flatnonzero(~seen.any(1))).cuda()
        for x, fill in ((k, float("nan")), (v, float("inf"))):
            x[i, gone] = fill
        q[i, blind] = float("nan")
        dout[i, blind] = float("-inf")
    d = torch.from_numpy(death.astype(np.int32)).cuda()
    out, lse = kvs.attend(q, k, v, d)
    grads = kvs.attend_backward(dout, q, k, v, out, lse, d)
    torch.cuda.synchronize()
    check(q, k, v, dout, death, dk ** -0.5, 0.0, out, lse, grads)
    # a value that some see: the others stay as they are, bit for bit or near
    v2 = v.clone()
    v2[0, at, head, 3] = float("inf")
    out2, lse2 = kvs.attend(q, k, v2, d)
    hit = W.death_seen(death[0])[:, at]
    o, o2 = f64(out), f64(out2)
    reached = np.zeros(out.shape, bool)
    reached[0, hit, head * G:(head + 1) * G, 3] = True
    assert not np.isfinite(o2[reached]).any()
    assert np.isfinite(o2[~reached]).all() and np.abs(o2 - o)[~reached].max() <= 4 * H * (1 + np.abs(o).max())
    assert torch.equal(torch.isfinite(lse), torch.isfinite(lse2))
    assert (lse - lse2)[torch.isfinite(lse)].abs().max() <= 1e-4
    # a query's gradient that is not finite: keys that it does not see stay finite
    dout2 = dout.clone()
    dout2[0, 120, head * G] = float("nan")
    grads2 = kvs.attend_backward(dout2, q, k, v, out, lse, d)
    sees = W.death_seen(death[0])[120]
    gv = f64(grads2[2])
    reached = np.zeros(v.shape, bool)
    reached[0, sees, head] = True
    assert np.isnan(gv[reached]).all() and np.isfinite(gv[~reached]).all()
    gk = f64(grads2[1])
    assert np.isfinite(gk[0, ~sees]).all() and np.isfinite(gk[1]).all() and np.isnan(gk[0, sees, head]).all()
    gq = f64(grads2[0])
    rest = np.ones(q.shape, bool)
    rest[0, 120, head * G] = False
    assert np.isfinite(gq[rest]).all() and np.isnan(gq[~rest]).all()
    # a key that is not finite: queries that do not see it keep their gradient
    k2 = k.clone()
    k2[0, at, head] = float("nan")
    out3, lse3 = kvs.attend(q, k2, v, d)
    grads3 = kvs.attend_backward(dout, q, k2, v, out3, lse3, d)
    gq = f64(grads3[0])
    rest = np.ones(q.shape, bool)
    rest[0, hit, head * G:(head + 1) * G] = False
    assert np.isfinite(gq[rest]).all() and np.isnan(gq[~rest]).all()
    kvs.close()


def test_scores_of_minus_infinity():
    """A query whose scores are all -inf gets zeros and no gradient."""
    L = need_gpu()
    kvs = L.KvsMask(0)
    g = np.random.default_rng(1)
    T = 80
    q, k, v = randn(g, 1, T, 1, 64).abs() + 1, randn(g, 1, T, 1, 64), randn(g, 1, T, 1, 64)
    k[0, :3] = float("-inf")
    dout = randn(g, 1, T, 1, 64)
    d = torch.full((1, T), T, dtype=torch.int32, device="cuda")
    out, lse = kvs.attend(q, k, v, d)
    dq, dk, dv = kvs.attend_backward(dout, q, k, v, out, lse, d)
    assert not out[0, :3].any() and torch.isneginf(lse[0, :3]).all() and torch.isfinite(lse[0, 3:]).all()
    assert torch.isfinite(out).all()
    assert not dq[0, :3].any() and torch.isfinite(dv).all() and not dv[0, :3].any()
    kvs.close()


def test_views_and_given_buffers():
    """One projection's output holds q, k and v; out, lse and the gradients go into
    parts of wider buffers, whose rest stays."""
    L = need_gpu()
    kvs = L.KvsMask(0)
    g = np.random.default_rng(2)
    n, T, Hk, G, D = 2, 150, 2, 3, 64
    heads = Hk * G
    x = randn(g, n, T + 3, heads + 2 * Hk, D)
    q, k, v = x[:, 2:T + 2, :heads], x[:, 2:T + 2, heads:heads + Hk], x[:, 2:T + 2, heads + Hk:]
    death = deaths("cut", n, T, g)
    d = torch.from_numpy(death.astype(np.int32)).cuda()
    wide = torch.full((n, heads, T + 1, 2 * D), 7.0, dtype=torch.bfloat16, device="cuda")   # head-major
    out = wide[:, :, 1:, D:].transpose(1, 2)
    lse = torch.zeros(n, T, heads, device="cuda")
    r = kvs.attend(q, k, v, d, out=out, lse=lse)
    assert r[0] is out and r[1] is lse
    dout = randn(g, n, heads, T, D).transpose(1, 2)
    gx = torch.full_like(x, 5.0)
    grads = (gx[:, 2:T + 2, :heads], gx[:, 2:T + 2, heads:heads + Hk], gx[:, 2:T + 2, heads + Hk:])
    back = kvs.attend_backward(dout, q, k, v, out, lse, d, grads=grads)
    torch.cuda.synchronize()
    check(q, k, v, dout, death, D ** -0.5, 0.0, out, lse, back)
    assert (wide[:, :, 0] == 7).all() and (wide[..., :D] == 7).all()
    assert (gx[:, :2] == 5).all() and (gx[:, T + 2:] == 5).all()
    # one key and value head for all through a stride of 0: a row of k's own gradient each
    kk, vv = k[:, :, :1].expand(n, T, heads, D), v[:, :, :1].expand(n, T, heads, D)
    out, lse = kvs.attend(q, kk, vv, d)
    back = kvs.attend_backward(dout, q, kk, vv, out, lse, d)
    check(q, kk, vv, dout, death, D ** -0.5, 0.0, out, lse, back)
    kvs.close()


def test_autograd_is_the_formulas_and_differences_agree():
    """attention() through torch's autograd against the same attention in float64 torch
    operations, and against differences of a loss along random directions."""
    L = need_gpu()
    kvs = L.KvsMask(0)
    g = np.random.default_rng(4)
    n, T, Hk, G, D = 1, 96, 1, 2, 64
    q, k, v = (randn(g, n, T, h, D).requires_grad_() for h in (Hk * G, Hk, Hk))
    death = deaths("cut", n, T, g)
    d = torch.from_numpy(death.astype(np.int32)).cuda()
    weight = randn(g, n, T, Hk * G, D)
    loss = (kvs.attention(q, k, v, d, cap=8.0) * weight).sum()
    loss.backward()
    seen = torch.from_numpy(W.death_seen(death[0])).cuda()

    def plain(q, k, v):
        x = torch.stack([q[0, :, h] @ k[0, :, h // G].t() for h in range(Hk * G)]) * D ** -0.5
        p = torch.softmax((8.0 * torch.tanh(x / 8.0)).masked_fill(~seen, float("-inf")), -1)
        return (torch.stack([p[h] @ v[0, :, h // G] for h in range(Hk * G)], 1) * weight[0].double()).sum()

    ref = [x.detach().double().requires_grad_() for x in (q, k, v)]
    plain(*ref).backward()
    for x, y in zip((q, k, v), ref):
        assert (x.grad.double() - y.grad).norm() <= 4 * H * y.grad.norm()
    for i in range(3):
        u = torch.randn(ref[i].shape, dtype=torch.float64, device="cuda")
        args = [x.detach() for x in ref]
        e = 1e-4
        hi = plain(*[a + e * u if j == i else a for j, a in enumerate(args)])
        lo = plain(*[a - e * u if j == i else a for j, a in enumerate(args)])
        diff = float(hi - lo) / (2 * e)
        got = float(((q, k, v)[i].grad.double() * u).sum())
        assert abs(got - diff) <= 4 * H * float(ref[i].grad.norm())   # |u| is near 1 in each direction
    # a broadcast gradient, and k alone
    k2 = k.detach().clone().requires_grad_()
    kvs.attention(q.detach(), k2, v.detach(), d).float().mean().backward()
    assert torch.isfinite(k2.grad).all() and k2.grad.any()
    kvs.close()


def test_same_bits_again_and_in_a_graph():
    """Forward and backward replayed in a graph, with new inputs and death times in the
    same buffers, give the eager call's bits; two graphs do not share a workspace."""
    L = need_gpu()
    kvs = L.KvsMask(0)
    g = np.random.default_rng(6)
    n, T, Hk, G, D = 1, 260, 2, 2, 128
    q, k, v = randn(g, n, T, Hk * G, D), randn(g, n, T, Hk, D), randn(g, n, T, Hk, D)
    dout = randn(g, n, T, Hk * G, D)
    d = torch.from_numpy(deaths("cut", n, T, g).astype(np.int32)).cuda()

    def both():
        out, lse = kvs.attend(q, k, v, d, cap=20.0)
        return (out, lse, *kvs.attend_backward(dout, q, k, v, out, lse, d, cap=20.0))

    first = [x.clone() for x in both()]
    assert all(torch.equal(a, b) for a, b in zip(first, both()))
    graphs, results = [], []
    for _ in range(2):
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.stream(s):
            with torch.cuda.graph(graph, stream=s):
                results.append(both())
        graphs.append(graph)
    for i in range(4):
        q.copy_(randn(g, *q.shape))
        d.copy_(torch.from_numpy(deaths(("cut", "doc", "any", "all")[i], n, T, g).astype(np.int32)))
        want = [x.clone() for x in both()]
        for r in results:
            for x in r:
                x.fill_(1)
        torch.cuda.synchronize()
        s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
        for graph, s in zip(graphs, (s1, s2)):
            with torch.cuda.stream(s):
                graph.replay()
        torch.cuda.synchronize()
        for r in results:
            assert all(torch.equal(a, b) for a, b in zip(want, r)), i
    with pytest.raises(RuntimeError):
        kvs_attention_captured(kvs, q, k, v, d)
    kvs.close()


def kvs_attention_captured(kvs, q, k, v, d):
    s = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(s):
        with torch.cuda.graph(graph, stream=s):
            q + 1
            kvs.attention(q, k, v, d)


def test_another_stream():
    """Results allocated for another stream's call, while the current one is busy."""
    L = need_gpu()
    kvs = L.KvsMask(0)
    g = np.random.default_rng(8)
    T, D = 300, 64
    q, k, v, dout = (randn(g, 1, T, 2, D) for _ in range(4))
    d = torch.full((1, T), T, dtype=torch.int32, device="cuda")
    out, lse = kvs.attend(q, k, v, d)
    want = kvs.attend_backward(dout, q, k, v, out, lse, d)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    out2, lse2 = kvs.attend(q, k, v, d, stream=s)
    got = kvs.attend_backward(dout, q, k, v, out2, lse2, d, stream=s)
    junk = [torch.full((1, T, 2, D), 3.0, dtype=torch.bfloat16, device="cuda") for _ in range(8)]
    s.synchronize()
    assert torch.equal(out, out2) and torch.equal(lse, lse2) and all(torch.equal(a, b) for a, b in zip(want, got))
    del junk
    kvs.close()


def test_refusals():
    L = need_gpu()
    kvs = L.KvsMask(0)
    z = lambda *s: torch.zeros(s, dtype=torch.bfloat16, device="cuda")   # noqa: E731
    q, k, v = z(1, 8, 4, 64), z(1, 8, 2, 64), z(1, 8, 2, 64)
    d = torch.full((1, 8), 8, dtype=torch.int32, device="cuda")
    out, lse = kvs.attend(q, k, v, d)
    for kw in (dict(k=z(1, 8, 3, 64), v=z(1, 8, 3, 64)), dict(q=z(1, 8, 4, 12), k=z(1, 8, 2, 12)), dict(v=z(1, 8, 2, 264)),
               dict(scale=float("nan")), dict(scale=float("inf")), dict(cap=-1.0), dict(cap=float("nan")),
               dict(cap=1e-30), dict(scale=1.0, cap=1e13), dict(scale=1e-25, cap=1e6),
               dict(out=z(1, 8, 1, 64).expand(1, 8, 4, 64)), dict(q=z(1, 8, 4, 68)[..., :64]),
               dict(q=z(1, 8, 1, 8 * 33 + 4)[..., 4:68].expand(1, 8, 4, 64))):
        with pytest.raises(L.LeylineError) as e:
            kvs.attend(**{"q": q, "k": k, "v": v, "death": d, **kw})
        assert e.value.status == L.LL_EINVAL, kw
    for kw in (dict(q=q.float()), dict(k=z(1, 7, 2, 64)), dict(v=v.cpu()), dict(death=d.long()), dict(death=d[0]),
               dict(death=torch.full((1, 9), 8, dtype=torch.int32, device="cuda")), dict(q=q[0]),
               dict(q=z(1, 8, 4, 128)[..., ::2]), dict(out=z(1, 8, 4, 32)), dict(lse=lse.double()),
               dict(lse=lse.transpose(1, 2)), dict(scale="x"), dict(k=None)):
        with pytest.raises(ValueError):
            kvs.attend(**{"q": q, "k": k, "v": v, "death": d, **kw})
    for kw in (dict(dout=z(1, 8, 4, 32)), dict(dout=out.float()), dict(out=None), dict(lse=None),
               dict(grads=(q, k, z(1, 8, 2, 32)))):
        with pytest.raises(ValueError):
            kvs.attend_backward(**{"dout": out, "q": q, "k": k, "v": v, "out": out, "lse": lse, "death": d, **kw})
    one = z(1, 8, 1, 64)
    with pytest.raises(L.LeylineError):
        kvs.attend_backward(out, q, k, v, out, lse, d, grads=(z(1, 8, 4, 64), one.expand(1, 8, 2, 64), z(1, 8, 2, 64)))
    # nothing to do
    e = lambda h, w: torch.zeros((0, 5, h, w), dtype=torch.bfloat16, device="cuda")   # noqa: E731
    d0 = torch.zeros((0, 5), dtype=torch.int32, device="cuda")
    o, l = kvs.attend(e(4, 64), e(2, 64), e(2, 64), d0)
    assert o.shape == (0, 5, 4, 64) and l.shape == (0, 5, 4)
    assert kvs.attend_backward(o, e(4, 64), e(2, 64), e(2, 64), o, l, d0)[1].shape == (0, 5, 2, 64)
    kvs.close()
