"""GPU parity of eviction by attention weight (include/leyline_weight.h) against the
float64 oracle, through the binding: capped attention and weighing over MLA and GQA
pools, single tokens to chunks, windows, odd sizes; selections with ties, NaN and
infinities, from one row to many.  Pool rows that no sequence holds are NaN.

Tolerances of the weights: a score is a float32 sum of dk products (dk 2^-24 of its
magnitudes), the exponent rounds score and lse a few times (8 2^-24 (1 + |s| + |lse|)), a
cap's tanh is off by 2^-21 of the score; each shifts its weight by that relatively.
exp2 is off by 2^-22, and a float32 sum of n of them by n 2^-24 at most."""

import numpy as np
import pytest

from oracle import weight_oracle as W

from gpu_common import need_gpu, say, torch
from test_gpu_step import ATTEND, Cache, F32, HALF_STEP, _cache, _queries, f64

pytestmark = pytest.mark.gpu


def check_capped(c, out, lse, q, seqs, counts, scale, cap, causal=True, window=0):
    worst, at = 0.0, 0
    got, gl, fq = f64(out), f64(lse), f64(q)
    heads = q.shape[1]
    for s, n in zip(seqs, counts):
        k = c.rows(0, 0, s)
        v = c.rows(1, 0, s) if c.gqa else k[..., :512]
        seen = W.step_seen(n, k.shape[0], k.shape[0] - n, causal, window)
        for h in range(heads):
            g = h // (heads // k.shape[1])
            o, l, w, slack = W.attend(fq[at:at + n, h], k[:, g], v[:, g], seen, scale, cap)
            ds = k.shape[-1] * F32 * slack + 8 * F32 * (1 + np.abs(l)) + 2.0 ** -21 * min(cap, slack.max(initial=0.0))
            tol = HALF_STEP * (np.abs(o) + w) + (2 * ds[:, None] + k.shape[0] * F32) * w + 1e-30
            bad = np.abs(got[at:at + n, h] - o) / tol
            assert np.isfinite(bad).all(), (s, h)
            worst = max(worst, float(bad.max(initial=0.0)))
            e = np.abs(gl[at:at + n, h] - l) / (ds + k.shape[0] * F32 + 1e-30)
            worst = max(worst, float(e.max(initial=0.0)))
            assert worst <= 1, (s, h, worst)
        at += n
    return worst


def weights_of(c, q, lse, seqs, counts, scale, cap, causal, window, heads):
    """Per sequence: (weights, tolerance) of the step."""
    fq, fl, at, res = f64(q), f64(lse), 0, []
    for s, n in zip(seqs, counts):
        k = c.rows(0, 0, s)
        rows, dk = k.shape[0], k.shape[-1]
        seen = W.step_seen(n, rows, rows - n, causal, window)
        total, tol = np.zeros(rows), np.zeros(rows)
        for h in range(heads):
            w, sl, x = W.weigh(fq[at:at + n, h], k[:, h // (heads // k.shape[1])], fl[at:at + n, h], seen, scale, cap)
            total += w
            tol += dk * F32 * sl + 8 * F32 * x + (2.0 ** -21 * x if cap else 0) + 2.0 ** -22 * w
        res.append((total, tol + (n * heads + 8) * F32 * total + 1e-37))
        at += n
    return res


@pytest.mark.parametrize("gqa,heads,kv_heads,dim,P,lens,counts", ATTEND)
@pytest.mark.parametrize("causal,window,cap", [(True, 0, 0.0), (True, 7, 4.0), (False, 0, 20.0)])
def test_capped_attention_and_weights(gqa, heads, kv_heads, dim, P, lens, counts, causal, window, cap):
    c = _cache(gqa, kv_heads, max(dim, 16), P, lens, seed=sum(lens))   # a band of 16 divides the head
    step = c.pool.step(heads, max_tokens=max(1, sum(counts)))
    T = step.begin(list(range(len(lens))), counts, grow=False)
    q = _queries(c, T, heads) * 2
    scale = 0.11
    seqs = list(range(len(lens)))
    out, lse = step.attend(0, q, scale=scale, causal=causal, window=window, lse=True, cap=cap)
    width = c.width * P + 5
    w = torch.full((len(lens), width), 0.5, device="cuda")
    got = step.weigh(0, q, lse, w, scale=scale, causal=causal, window=window, cap=cap, decay=0.25)
    assert got is w
    torch.cuda.synchronize()
    worst = check_capped(c, out, lse, q, seqs, counts, scale, cap, causal, window) if cap else 0.0
    far = 0.0
    for i, (want, tol) in enumerate(weights_of(c, q, lse, seqs, counts, scale, cap, causal, window, heads)):
        e = np.abs(w[i, :lens[i]].double().cpu().numpy() - (want + 0.125)) / (tol + 2 * F32 * (want + 0.125))
        far = max(far, float(e.max(initial=0.0)))
        assert far <= 1, (i, far, int(e.argmax()))
        assert (w[i, lens[i]:] == 0.5).all()
    say(f"attend {worst:.2f} weigh {far:.2f}")
    # what was there, NaN too, counts nothing at decay 0; twice the same bits
    a = torch.full_like(w, float("nan"))
    step.weigh(0, q, lse, a, scale=scale, causal=causal, window=window, cap=cap, decay=0.0)
    b = torch.zeros_like(w)
    step.weigh(0, q, lse, b, scale=scale, causal=causal, window=window, cap=cap, decay=0.0)
    for i, n in enumerate(lens):
        assert torch.equal(a[i, :n], b[i, :n]) and torch.isnan(a[i, n:]).all()
    if causal and not window:
        for i, n in enumerate(counts):
            total = float(b[i, :lens[i]].double().sum())
            assert abs(total - n * heads) <= 1e-4 * max(1, n * heads)
    step.close()
    c.pool.close()


@pytest.mark.parametrize("gqa", [False, True])
@pytest.mark.parametrize("n,count", [(5000, 1), (20011, 3), (3000, 700), (1700, 1700)])
def test_long_sequences(gqa, n, count):
    """Several tiles of rows and of queries, another sequence beside it that is not in
    the step."""
    heads = 16
    c = _cache(gqa, 4, 64, 16, [n, 40], seed=n)
    step = c.pool.step(heads, max_tokens=count)
    T = step.begin([0], [count], grow=False)
    q = _queries(c, T, heads)
    out, lse = step.attend(0, q, scale=0.1, lse=True, cap=6.0)
    w = torch.zeros(2, n + 3, device="cuda")
    step.weigh(0, q, lse, w, scale=0.1, cap=6.0)
    step.weigh(0, q, lse, w, scale=0.1, cap=6.0)
    (want, tol), = weights_of(c, q, lse, [0], [count], 0.1, 6.0, True, 0, heads)
    e = np.abs(w[0, :n].double().cpu().numpy() - 2 * want) / (2 * tol + 2 * F32 * want)
    assert e.max() <= 1, (float(e.max()), int(e.argmax()))
    assert not w[1].any() and not w[0, n:].any()
    assert check_capped(c, out, lse, q, [0], [count], 0.1, 6.0) <= 1
    step.close()
    c.pool.close()


@pytest.mark.parametrize("gqa", [False, True])
def test_caps_and_scales_at_their_ends(gqa):
    c = _cache(gqa, 2, 64, 16, [150], seed=3)
    step = c.pool.step(4, max_tokens=20)
    step.begin([0], [20], grow=False)
    q = _queries(c, 20, 4)
    for scale, cap in ((0.0, 3.0), (-0.5, 3.0), (2.0, 2.0 ** -40), (1.0, 2.0 ** 40), (30.0, 50.0), (2.0 ** -30, 2.0 ** 30)):
        out, lse = step.attend(0, q, scale=scale, lse=True, cap=cap)
        assert check_capped(c, out, lse, q, [0], [20], scale, cap) <= 1, (scale, cap)
        w = torch.zeros(1, 150, device="cuda")
        step.weigh(0, q, lse, w, scale=scale, cap=cap)
        (want, tol), = weights_of(c, q, lse, [0], [20], scale, cap, True, 0, 4)
        assert (np.abs(w[0].double().cpu().numpy() - want) <= tol + F32 * want).all(), (scale, cap)
    same = step.attend(0, q, scale=0.1)
    assert torch.equal(same, step.attend(0, q, scale=0.1, cap=0.0))
    step.close()
    c.pool.close()


@pytest.mark.parametrize("gqa", [False, True])
def test_values_that_are_not_finite(gqa):
    """NaN and infinities in rows that a token does not see change nothing; a token whose
    scores are all -inf adds nothing; under a cap such a score counts -cap."""
    c = _cache(gqa, 2, 64, 16, [90], seed=5)
    heads = 4
    step = c.pool.step(heads, max_tokens=30)
    step.begin([0], [30], grow=False)
    q = _queries(c, 30, heads).abs() + 0.5
    w0 = torch.zeros(1, 90, device="cuda")
    _, lse = step.attend(0, q, scale=0.1, lse=True, window=20)
    step.weigh(0, q, lse, w0, scale=0.1, window=20)
    for x in c.planes:
        x[0].view(-1, *x.shape[3:])[c.slots(0, 0, 41)] = float("nan")    # the first token sees rows 41 on
    w1 = torch.zeros(1, 90, device="cuda")
    out, lse1 = step.attend(0, q, scale=0.1, lse=True, window=20)
    assert torch.isfinite(out).all() and torch.isfinite(lse1).all()
    step.weigh(0, q, lse, w1, scale=0.1, window=20)
    assert torch.equal(w0, w1)
    k = c.planes[0][0].view(-1, *c.planes[0].shape[3:])
    k[c.slots(0, 41, 90)] = float("-inf")
    out, lse = step.attend(0, q, scale=0.1, lse=True, window=20)
    assert torch.isneginf(lse).all()
    step.weigh(0, q, lse, w1, scale=0.1, window=20, decay=0.5)
    assert torch.equal(w1, w0 * 0.5)
    out, lse = step.attend(0, q, scale=0.1, lse=True, window=20, cap=5.0)
    assert (lse - (np.log(20) - 5)).abs().max() <= 1e-5
    step.weigh(0, q, lse, w1, scale=0.1, window=20, cap=5.0, decay=0.0)
    assert not w1[0, :41].any() and abs(float(w1.sum()) - 30 * heads) <= 1e-3
    step.close()
    c.pool.close()


@pytest.mark.parametrize("gqa", [False, True])
def test_weigh_in_a_graph(gqa):
    """A captured weighing follows later begins, other lengths and counts among them."""
    heads, P = 8, 16
    lens = [70, 33, 200]
    c = _cache(gqa, 2, 64, P, lens, seed=9, room=200)
    step = c.pool.step(heads, max_seqs=3, max_tokens=40)
    step.begin([0, 1, 2], [1, 1, 1], grow=False)
    q = _queries(c, 40, heads)
    out, lse = torch.zeros(40, heads, 512 if not gqa else 64, dtype=torch.bfloat16, device="cuda"), torch.zeros(40, heads, device="cuda")
    w = torch.zeros(3, c.width * P, device="cuda")

    def both(weights):
        step.attend(0, q, scale=0.1, out=out, lse=lse, cap=9.0)
        step.weigh(0, q, lse, weights, scale=0.1, cap=9.0, decay=0.5)

    both(w)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(s):
        with torch.cuda.graph(graph, stream=s):
            both(w)
        with pytest.raises(c.L.LeylineError):
            with torch.cuda.graph(torch.cuda.CUDAGraph(), stream=s):
                step.weigh(0, q, lse, torch.zeros(3, 200, device="cuda"), scale=0.1)
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        for seqs, counts in (([0, 1, 2], [1, 1, 1]), ([2], [33]), ([1, 0], [0, 5]), ([0, 1, 2], [3, 20, 1])):
            step.begin(seqs, counts, grow=False)
            want = torch.rand(3, c.width * P, device="cuda")
            w.copy_(want)
            both(want)
            got_lse = lse.clone()
            lse.fill_(3)
            graph.replay()
            torch.cuda.synchronize()
            # the graph keeps its tiles, whose sums go in another order
            T = sum(counts)
            assert (lse[:T] - got_lse[:T]).abs().max() <= 1e-5 and (lse[T:] == 3).all(), (seqs, counts)
            gone = torch.ones(w.shape, dtype=torch.bool, device="cuda")
            for i in seqs:
                gone[i, :lens[i]] = False
            assert torch.equal(w[gone], want[gone]), (seqs, counts)
            assert ((w - want).abs() <= 1e-4 * (0.01 + want)).all(), (seqs, counts)
    step.close()
    c.pool.close()


def test_far_rows_of_a_long_sequence():
    """Rows past 2^20 of a cache of more than 2^32 bytes, weights past 2^31 bytes."""
    L = need_gpu()
    n, H, D, P, heads = (1 << 20) + 77, 8, 256, 256, 8
    pages = -(-n // P)
    k = torch.zeros(1, pages, P, H, D, dtype=torch.bfloat16, device="cuda")
    k.view(-1, H, D)[n - 300:n] = torch.randn(300, H, D, device="cuda").bfloat16()
    v = k.clone()
    table = torch.full((520, pages), -1, dtype=torch.int32, device="cuda")
    pool = L.GqaPool(k, v, table, rotary_dim=64)
    last = 515
    pool.seq_set_pages(last, np.arange(pages)[::-1].copy(), n)
    k.view(-1, P, H, D)[:] = k.view(-1, P, H, D).flip(0).clone()
    step = pool.step(heads, max_seqs=1, max_tokens=2)
    step.begin([last], [2], grow=False)
    q = torch.randn(2, heads, D, device="cuda").bfloat16()
    out, lse = step.attend(0, q, lse=True)
    w = torch.zeros(520, pages * P, device="cuda")
    step.weigh(0, q, lse, w)
    torch.cuda.synchronize()
    rows = k[0].flip(0).reshape(-1, H, D)[:n]
    want = torch.zeros(n, dtype=torch.float64, device="cuda")
    for t in range(2):
        for h in range(heads):
            x = (rows[:n - 1 + t, h].float() @ q[t, h].float()) * D ** -0.5
            want[:n - 1 + t] += (x.double() - lse[t, h].double()).exp()
    assert (w[last, :n].double() - want).abs().max() <= 1e-5 * want.max() and abs(float(w.double().sum()) - 16) <= 1e-3
    assert not w[:last].any() and not w[last, n:].any()
    keep, off = pool.keep_heaviest([last], [300], w, sinks=2, recent=3, kept_weights=w)
    assert list(off) == [0] and int(keep.sum()) == 300 and keep[:2].all() and keep[n - 3:].all()
    assert torch.equal(torch.nonzero(w[last]).flatten()[-1:].cpu() < 300, torch.tensor([True]))
    step.close()
    pool.close()


# ---- selections

def make(g, n, kind):
    w = np.exp(2 * g.standard_normal(n)).astype(np.float32)
    if kind == "ties":
        w = g.integers(0, 3, n).astype(np.float32)
    elif kind == "zeros":
        w[:] = 0
        w[::3] = -0.0
    elif kind == "odd":
        w[g.random(n) < 0.1] = np.nan
        w[g.random(n) < 0.1] = np.inf
        w[g.random(n) < 0.1] = -np.inf
        w[g.random(n) < 0.1] = np.finfo(np.float32).min
        w[g.random(n) < 0.1] = 1e-42
        w = np.where(g.random(n) < 0.3, -w, w).astype(np.float32)
    elif kind == "near":     # the last bits decide
        w = (np.float32(1) + g.integers(0, 300, n) * np.float32(2.0 ** -23)).astype(np.float32)
    return w


@pytest.mark.parametrize("kind", ["spread", "ties", "zeros", "odd", "near"])
@pytest.mark.parametrize("lens,sinks,recent", [([1], 0, 0), ([1, 2, 63, 64, 65], 1, 1), ([1023, 1024, 1025], 4, 16),
                                               ([8191, 8192, 8193, 300], 3, 100), ([40000, 7], 4, 64), ([131079], 0, 1000)])
def test_selection(kind, lens, sinks, recent):
    L = need_gpu()
    P = 16
    g = np.random.default_rng(len(lens) + lens[0])
    cache = torch.zeros(1, sum(-(-n // P) for n in lens) + 1, P, 576, dtype=torch.bfloat16, device="cuda")
    table = torch.full((len(lens) + 2, -(-max(lens) // P)), -1, dtype=torch.int32, device="cuda")
    pool = L.Pool(cache, table)
    pool.seq_alloc(0)
    for n in lens:
        pool.seq_alloc(n)
    room = -(-max(lens) // P) * P + 3
    host = np.full((len(lens) + 2, room), 9.0, np.float32)
    for i, n in enumerate(lens):
        host[i + 1, :n] = make(g, n, kind)
    w = torch.from_numpy(host).cuda()
    order = [int(x) for x in g.permutation(len(lens))]
    for share in (0.0, 0.3, 0.9, 1.0, 2.0):
        budgets = [max(int(lens[i] * share), sinks + recent) for i in order]
        out = torch.full_like(w, 5.0)
        seqs = [i + 1 for i in order]
        keep, off = pool.keep_heaviest(seqs, budgets, w, sinks=sinks, recent=recent, kept_weights=out)
        inplace = w.clone()
        keep2, _ = pool.keep_heaviest(seqs, budgets, inplace, sinks=sinks, recent=recent, kept_weights=inplace)
        torch.cuda.synchronize()
        assert torch.equal(keep, keep2)
        got, moved, moved2 = keep.cpu().numpy(), out.cpu().numpy(), inplace.cpu().numpy()
        for s, b, o in zip(seqs, budgets, off):
            n = lens[s - 1]
            want = W.keep_heaviest(host[s, :n], b, sinks, recent)
            assert np.array_equal(got[o:o + n], want), (s, b, np.flatnonzero(got[o:o + n] != want)[:5])
            exp = np.full(room, 5.0, np.float32)
            exp[:n] = 0
            exp[:want.sum()] = host[s, :n][want == 1]
            np.testing.assert_array_equal(moved[s], exp)
            exp[n:] = 9.0
            np.testing.assert_array_equal(moved2[s], exp)
        assert (moved[0] == 5).all() and (moved2[0] == 9).all() and (moved[-1] == 5).all()
        # the eviction takes the mask as it is
    n0 = pool.seq_get(seqs[0])[0]
    pool.evict(seqs, keep, off)
    assert pool.seq_get(seqs[0])[0] == min(budgets[0], n0)
    pool.close()


def test_many_sequences_and_a_given_mask():
    """More sequences than one launch takes, an empty one among them; the mask goes into
    a wider buffer."""
    L = need_gpu()
    g = np.random.default_rng(0)
    lens = [int(x) for x in g.integers(1, 200, 250)]
    lens[7] = 0
    cache = torch.zeros(1, sum(-(-n // 4) for n in lens), 4, 576, dtype=torch.bfloat16, device="cuda")
    pool = L.Pool(cache, torch.full((250, 50), -1, dtype=torch.int32, device="cuda"))
    for n in lens:
        pool.seq_alloc(n)
    host = g.random((250, 200)).astype(np.float32)
    buf = torch.full((sum(lens) + 9,), 7, dtype=torch.uint8, device="cuda")
    keep, off = pool.keep_heaviest(list(range(250)), [50] * 250, torch.from_numpy(host).cuda(), keep=buf)
    assert keep is buf
    got = buf.cpu().numpy()
    for i, n in enumerate(lens):
        assert np.array_equal(got[off[i]:off[i] + n], W.keep_heaviest(host[i, :n], 50, 0, 0)), i
    assert (got[sum(lens):] == 7).all()
    pool.close()


def test_refusals():
    L = need_gpu()
    c = _cache(True, 2, 64, 16, [50, 20], seed=1)
    step = c.pool.step(4, max_tokens=8)
    q, w = _queries(c, 8, 4), torch.zeros(2, 64, device="cuda")
    lse = torch.zeros(8, 4, device="cuda")
    with pytest.raises(L.LeylineError):
        step.weigh(0, q, lse, w)             # no begin yet
    step.begin([0], [8], grow=False)
    step.weigh(0, q, lse, w)
    for kw in (dict(layer=1), dict(layer=-1), dict(window=-1), dict(window=3, causal=False), dict(scale=float("nan")),
               dict(cap=-1.0), dict(cap=float("inf")), dict(cap=1e-20), dict(cap=1e13), dict(decay=-0.1), dict(decay=1.5),
               dict(decay=float("nan")), dict(weights=torch.zeros(2, 49, device="cuda"))):
        with pytest.raises(L.LeylineError) as e:
            step.weigh(**{"layer": 0, "q": q, "lse": lse, "weights": w, **kw})
        assert e.value.status == L.LL_EINVAL, kw
    for cap, scale in ((-1.0, 1.0), (float("nan"), 1.0), (float("inf"), 1.0), (1e-20, 1.0), (1e13, 1.0), (1e10, 1e-12),
                       (1e-10, 1e10)):
        with pytest.raises(L.LeylineError) as e:
            step.attend(0, q, scale=scale, cap=cap)
        assert e.value.status == L.LL_EINVAL
    for kw in (dict(weights=w.double()), dict(weights=w[:1]), dict(weights=w.t()), dict(weights=w.cpu()),
               dict(weights=torch.zeros(2, 128, device="cuda")[:, ::2]), dict(lse=lse.t().contiguous()),
               dict(lse=lse.bfloat16()), dict(decay="x"), dict(cap="x"), dict(q=q.float()), dict(lse=None)):
        with pytest.raises(ValueError):
            step.weigh(**{"layer": 0, "q": q, "lse": lse, "weights": w, **kw})
    with pytest.raises(ValueError):
        step.attend(0, q, cap="x")
    for kw in (dict(seqs=[5]), dict(seqs=[0, 0], budgets=[20, 20]), dict(budgets=[-1]), dict(budgets=[9], sinks=5, recent=5),
               dict(sinks=-1), dict(recent=-1), dict(weights=torch.zeros(2, 49, device="cuda"))):
        with pytest.raises(L.LeylineError) as e:
            c.pool.keep_heaviest(**{"seqs": [0], "budgets": [20], "weights": w, **kw})
        assert e.value.status == L.LL_EINVAL, kw
    for kw in (dict(budgets=[1, 2]), dict(keep=torch.zeros(49, dtype=torch.uint8, device="cuda")),
               dict(keep=torch.zeros(50, device="cuda")), dict(kept_weights=w.double()), dict(weights=w.cpu()),
               dict(kept_weights=torch.zeros(2, 65, device="cuda")), dict(weights=np.zeros((2, 64), np.float32))):
        with pytest.raises(ValueError):
            c.pool.keep_heaviest(**{"seqs": [0], "budgets": [20], "weights": w, **kw})
    buf = torch.zeros(3, 64, device="cuda")
    with pytest.raises(L.LeylineError):      # neither the same buffer nor another one
        c.pool.keep_heaviest([0, 1], [20, 20], buf[:2], kept_weights=buf[1:])
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        with pytest.raises(L.LeylineError) as e:
            with torch.cuda.graph(torch.cuda.CUDAGraph(), stream=s):
                c.pool.keep_heaviest([0], [20], w)
        assert e.value.status == L.LL_EUNSUPPORTED
    torch.cuda.synchronize()
    assert c.pool.keep_heaviest([], [], w)[0].numel() == 0
    c.pool.evict([0], c.pool.keep_heaviest([0], [20], w)[0], [0])
    with pytest.raises(L.LeylineError):      # the sequence has changed since the step began
        step.weigh(0, q, lse, w)
    step.close()
    c.pool.close()
