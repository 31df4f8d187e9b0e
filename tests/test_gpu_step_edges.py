"""The serving step where it can go wrong, on the GPU against the float64 oracle:
values that are not finite in rows that a token does not see, scores far apart,
every tile size and long splits, growth between splices, evictions and frees,
captured and replayed steps, other streams, views and spare buffer rows, offsets
past 32 bits, page tables that something else has overwritten.  Tolerances are
those of test_gpu_step.py unless a test derives its own."""

import numpy as np
import pytest

from oracle import step_oracle as S

from gpu_common import need_gpu, say, torch
from test_gpu_step import F32, HALF_STEP, Cache, _cache, _queries, bf16, f64

pytestmark = pytest.mark.gpu

INF, NAN = float("inf"), float("nan")
LOWEST = -3.3895313892515355e38   # bf16's


def plant(c, plane, layer, seq, row, cols, value):
    x = c.planes[plane][layer]
    x = x.view(-1, *x.shape[2:])
    x[c.slots(seq, row, row + 1), ..., cols] = value


@pytest.mark.parametrize("kind", ["mla", "gqa64", "gqa96", "gqa256"])
@pytest.mark.parametrize("value", [NAN, INF, -INF, LOWEST])
@pytest.mark.parametrize("window", [0, 40])
def test_unseen_rows_never_reach_a_result(kind, value, window):
    """A chunk whose later rows (seen by some of its tokens only), and rows before
    every window, hold such values: tokens that do not see them get what they would
    get, tokens that see a NaN get NaN where the formula does."""
    gqa, dim = kind != "mla", int(kind[3:] or 0) if kind != "mla" else 576
    heads, kv = (4, 2) if gqa else (8, 1)
    n, count = 137, 50
    c = _cache(gqa, kv, dim, 16, [n], seed=3)
    first = n - count
    spots = [first + 20, first + 49] + ([5, 30] if window else [])   # the window starts at row 48 at the earliest
    for r in spots:
        for plane in range(len(c.planes)):
            plant(c, plane, 0, 0, r, slice(None) if r != first + 20 else slice(3, 4), value)
    step = c.pool.step(heads, max_tokens=count)
    step.begin([0], [count], grow=False)
    q = _queries(c, count, heads)
    out, lse = step.attend(0, q, scale=0.06, window=window, lse=True)
    torch.cuda.synchronize()
    got, gl, ql = f64(out), f64(lse), f64(q)
    k = c.rows(0, 0, 0)
    v = c.rows(1, 0, 0) if gqa else k[..., :512]
    clean = 20   # tokens before first + 20 see none of it
    for h in range(heads):
        x = h // (heads // k.shape[1])
        with np.errstate(all="ignore"):
            o, l, w, slack = S.attend(ql[:, h], k[:, x], v[:, x], first, 0.06, True, window)
        tol = HALF_STEP * (np.abs(o) + w) + (2 * k.shape[-1] * F32 * slack[:, None] + 16 * F32 * (1 + np.abs(l[:, None])) + n * F32) * w
        assert np.isfinite(o[:clean]).all()
        assert (np.abs(got[:clean, h] - o[:clean]) <= tol[:clean]).all(), h
        assert np.isfinite(gl[:clean, h]).all()
        if np.isnan(value):
            assert np.array_equal(np.isnan(got[:, h]), np.isnan(o)), h
            assert np.array_equal(np.isnan(gl[:, h]), np.isnan(l)), h
    step.close()
    c.pool.close()


@pytest.mark.parametrize("gqa", [False, True])
@pytest.mark.parametrize("causal", [True, False])
def test_visible_values_that_are_not_finite(gqa, causal):
    """One token over many rows, NaN in one column of a value: as the formula (MLA:
    the value is part of the key, so all of it)."""
    c = _cache(gqa, 1, 64 if gqa else 576, 4, [300, 300], seed=4)
    plant(c, 1 if gqa else 0, 0, 0, 100, slice(7, 8), NAN)
    step = c.pool.step(2, max_tokens=2)
    step.begin([0, 1], [1, 1], grow=False)
    q = _queries(c, 2, 2)
    got = f64(step.attend(0, q, scale=0.1, causal=causal))
    assert np.isfinite(got[1]).all() and np.isnan(got[0, :, 7]).all()
    if gqa:
        assert np.isfinite(np.delete(got[0], 7, 1)).all()
    else:
        assert np.isnan(got[0]).all()
    step.close()
    c.pool.close()


@pytest.mark.parametrize("scale", [8.0, -8.0, 0.25, 0.0, 1e-30])
@pytest.mark.parametrize("count", [1, 33, 140])
@pytest.mark.parametrize("gqa", [False, True])
def test_scores_far_apart(gqa, count, scale):
    """Keys that grow along the sequence (the running maximum moves at every tile)
    and queries with one value: products are exact, and a score s is off by its
    rounded factors only, at most 4 F32 |s|; a weight by the difference of two."""
    n = 400
    c = _cache(gqa, 1, 128 if gqa else 576, 16, [n], seed=6)
    x = c.planes[0][0]
    x = x.view(-1, *x.shape[2:])
    ramp = bf16(np.linspace(-60, 60, n)).cuda()
    s = c.slots(0, 0, n)
    x[s, ..., 5] = ramp[:, None] if gqa else ramp
    heads = 3
    q = torch.zeros((count, heads, 128 if gqa else 576), dtype=torch.bfloat16, device="cuda")
    for h, v in enumerate((1.0, -2.0, 8.0)):
        q[:, h, 5] = v
    step = c.pool.step(heads, max_tokens=count)
    step.begin([0], [count], grow=False)
    out, lse = step.attend(0, q, scale=scale, lse=True)
    got, gl = f64(out), f64(lse)
    k = c.rows(0, 0, 0)[:, 0]
    v = c.rows(1, 0, 0)[:, 0] if gqa else k[:, :512]
    for h in range(heads):
        o, l, w, slack = S.attend(f64(q)[:, h], k, v, n - count, scale)
        ds = 4 * F32 * slack[:, None] + 8 * F32 * (1 + np.abs(l[:, None]))
        assert (np.abs(got[:, h] - o) <= HALF_STEP * (np.abs(o) + w) + (2 * ds + n * F32) * w).all(), h
        assert (np.abs(gl[:, h] - l) <= ds[:, 0] + n * F32).all(), h
    step.close()
    c.pool.close()


@pytest.mark.parametrize("kind", ["mla", "gqa64", "gqa96", "gqa128", "gqa256"])
@pytest.mark.parametrize("count", [3, 8, 13, 30, 70])
def test_every_tile_size(kind, count):
    """12, 32, 52, 120 and 280 query rows: the tiles of 16 to 256; a sequence whose
    rows end inside a tile, one that is all chunk."""
    gqa, dim = kind != "mla", int(kind[3:]) if kind != "mla" else 576
    c = _cache(gqa, 2, dim, 16, [count + 210, count], seed=count)
    heads = 8 if gqa else 4
    step = c.pool.step(heads, max_tokens=2 * count)
    T = step.begin([0, 1], [count, count], grow=False)
    q = _queries(c, T, heads)
    for kw in (dict(), dict(window=33), dict(causal=False)):
        out, lse = step.attend(0, q, scale=0.08, lse=True, **kw)
        c.check_attend(out, lse, q, [0, 1], [count, count], 0, 0.08, kw.get("causal", True), kw.get("window", 0))
    step.close()
    c.pool.close()


@pytest.mark.parametrize("dim", [16, 48, 80, 112, 144, 192, 240])
@pytest.mark.parametrize("count", [1, 9, 45])
def test_head_widths_between_the_powers_of_two(dim, count):
    c = _cache(True, 2, dim, 16, [170, count], seed=dim)
    step = c.pool.step(6, max_tokens=2 * count)
    T = step.begin([1, 0], [count, count], grow=False)
    q = _queries(c, T, 6)
    out, lse = step.attend(0, q, lse=True)
    c.check_attend(out, lse, q, [1, 0], [count, count], 0, dim ** -0.5)
    step.close()
    c.pool.close()


@pytest.mark.parametrize("gqa", [False, True])
def test_queries_or_rows_alone(gqa):
    """append without rows or without queries does that part of the whole call."""
    c = Cache(gqa, 16, [50], seed=5, kv_heads=2, dim=64, rot=64, room=20)
    step = c.pool.step(5 if not gqa else 6, max_tokens=9)
    T = step.begin([0], [9])
    g = np.random.default_rng(4)
    a = bf16(g.standard_normal((T, 2, 64) if gqa else (T, 512))).cuda()
    b = bf16(g.standard_normal((T, 2, 64) if gqa else (T, 64))).cuda()
    q = bf16(g.standard_normal((T, 6 if gqa else 5, 64))).cuda()
    both = step.append(0, a, b, q=q)
    rows = [c.rows(p, 0, 0, 50) for p in range(len(c.planes))]
    for p in range(len(c.planes)):
        plant(c, p, 0, 0, 55, slice(None), 3.0)
    assert torch.equal(step.append(0, q=q), both)
    assert not np.array_equal(c.rows(0, 0, 0, 50), rows[0])   # no row was written
    assert step.append(0, a, b) is None
    for p in range(len(c.planes)):
        assert np.array_equal(c.rows(p, 0, 0, 50), rows[p])
    step.close()
    c.pool.close()


@pytest.mark.parametrize("gqa", [False, True])
@pytest.mark.parametrize("P", [1, 16])
def test_a_begin_right_behind_an_eviction(gqa, P):
    """Nothing reads the sequence in between: at page size 1 its length is still on
    the device."""
    c = Cache(gqa, P, [300, 40], seed=P, kv_heads=2, dim=64, rot=64, room=40, spare=-(-360 // P) + 4)
    step = c.pool.step(4, max_tokens=8)
    g = np.random.default_rng(6)
    keep = (g.random(300) > 0.4).astype(np.uint8)
    want = [c.rows(p, 0, 0)[keep == 1] for p in range(len(c.planes))]
    mask = torch.from_numpy(keep).cuda()
    q = _queries(c, 5, 4)
    a = bf16(g.standard_normal((5, 2, 64) if gqa else (5, 512))).cuda()
    b = bf16(g.standard_normal((5, 2, 64) if gqa else (5, 64))).cuda()
    c.pool.evict([0], mask, [0])
    step.begin([0, 1], [3, 2])
    step.append(0, a, b)
    out, lse = step.attend(0, q, scale=0.1, lse=True)
    torch.cuda.synchronize()
    n = int(keep.sum())
    assert c.pool.seq_get(0)[:2] == (n + 3, 303)
    for p in range(len(c.planes)):
        assert np.array_equal(c.rows(p, 0, 0, 0, n), want[p])
    c.check_attend(out, lse, q, [0, 1], [3, 2], 0, 0.1)
    step.close()
    c.pool.close()


@pytest.mark.parametrize("gqa,heads,kv,dim,P,lens,counts,window", [
    (False, 16, 1, 576, 64, [40007], [1], 0),
    (False, 8, 1, 576, 16, [9000, 5, 20001], [1, 1, 2], 0),
    (False, 16, 1, 576, 16, [6001], [9], 2500),
    (True, 8, 2, 128, 16, [30011], [1], 0),
    (True, 4, 1, 64, 1, [7003, 1, 2], [5, 1, 2], 0),
    (True, 4, 2, 256, 256, [12001], [2], 6000),
])
def test_long_sequences_split_and_joined(gqa, heads, kv, dim, P, lens, counts, window):
    say(f"long gqa={gqa} dim={dim} lens={lens} counts={counts} window={window}")
    c = _cache(gqa, kv, dim, P, lens, seed=len(lens))
    step = c.pool.step(heads, max_tokens=16)
    seqs = list(range(len(lens)))
    T = step.begin(seqs, counts, grow=False)
    q = _queries(c, T, heads)
    out, lse = step.attend(0, q, scale=0.05, window=window, lse=True)
    again = step.attend(0, q, scale=0.05, window=window)
    assert torch.equal(out.view(torch.int16), again.view(torch.int16))
    c.check_attend(out, lse, q, seqs, counts, 0, 0.05, True, window)
    step.close()
    c.pool.close()


def test_a_far_position_and_a_million_rows():
    """A sequence of 2^20 + 5 narrow rows: positions past 2^20 in append, and one
    token's attention over all of them."""
    n = (1 << 20) + 5
    c = Cache(True, 256, [n], kv_heads=1, dim=16, rot=16, pairing=1, room=300, base=500000.0)
    step = c.pool.step(2, max_tokens=4)
    T = step.begin([0], [3])
    g = np.random.default_rng(1)
    a, b, q = (bf16(g.standard_normal((T, h, 16))).cuda() for h in (1, 1, 2))
    ang = S.angles(n + np.arange(3), 16, 500000.0)
    qo = step.append(0, a, b, q=q)
    want, size = S.heads(f64(a), None, 0, ang, 1, 16)
    c.check_rows(0, 0, 0, n, n + 3, want, size)
    want, size = S.heads(f64(q), None, 0, ang, 1, 16)
    assert (np.abs(f64(qo) - want) <= HALF_STEP * np.abs(want) + 2.0 ** -18 * size).all()
    out, lse = step.attend(0, qo, lse=True)
    c.check_attend(out, lse, qo, [0], [3], 0, 0.25)
    step.close()
    c.pool.close()


def _layer(c, step, layer, T, heads, g, check):
    """Append and attend one layer with random inputs; check is told what came out."""
    dq = c.D if c.gqa else 64
    if c.gqa:
        a, b = (bf16(g.standard_normal((T, c.H, c.D))).cuda() for _ in range(2))
        lat = None
    else:
        a, b = bf16(g.standard_normal((T, 512))).cuda(), bf16(g.standard_normal((T, 64))).cuda()
        lat = bf16(g.standard_normal((T, heads, 512))).cuda()
    q = bf16(g.standard_normal((T, heads, dq))).cuda()
    asked = q.clone()
    w = bf16(1 + 0.1 * g.standard_normal(c.D if c.gqa else 512)).cuda()
    assert step.append(layer, a, b, norm=w, q=q, q_out=q, eps=1e-6) is q   # in place
    if c.gqa:
        out, lse = step.attend(layer, q, lse=True)
    else:
        out, lse = step.attend(layer, lat, q, scale=0.05, lse=True)
    check(layer, a, b, w, asked, q, lat, out, lse)


def _run_step(c, step, seqs, counts, heads, g, layers):
    before = {s: c.pool.seq_get(s)[:2] for s in seqs}
    T = step.begin(seqs, counts)
    assert T == sum(counts)
    pos = np.concatenate([before[s][1] + np.arange(n) for s, n in zip(seqs, counts)]) if T else np.zeros(0)
    ang = S.angles(pos, c.rot if c.gqa else 64, c.base)

    def check(layer, a, b, w, asked, q, lat, out, lse):
        ww = f64(w)
        want, size = S.heads(f64(asked), None, 0, ang, c.pairing, c.rot if c.gqa else 64)
        assert (np.abs(f64(q) - want) <= HALF_STEP * np.abs(want) + 2.0 ** -18 * size).all()
        lo = 0
        for s, n in zip(seqs, counts):
            at, sl = before[s][0], slice(lo, lo + n)
            if c.gqa:
                c.check_rows(0, layer, s, at, at + n, *S.heads(f64(a[sl]), ww, 1e-6, ang[sl], c.pairing, c.rot))
                assert np.array_equal(c.rows(1, layer, s, at, at + n), f64(b[sl]))
            else:
                latent = S.norm(f64(a[sl])[:, None], ww, 1e-6)
                pe, sp = S.heads(f64(b[sl])[:, None], None, 0, ang[sl], c.pairing)
                c.check_rows(0, layer, s, at, at + n, np.concatenate([latent, pe], -1),
                             np.concatenate([np.abs(latent), sp], -1))
            lo += n
        full = q if c.gqa else torch.cat([lat, q], -1)
        c.check_attend(out, lse, full, seqs, counts, layer, c.D ** -0.5 if c.gqa else 0.05)

    for layer in range(layers):
        _layer(c, step, layer, T, heads, g, check)


@pytest.mark.parametrize("gqa,P,pairing", [(False, 1, 0), (False, 16, 1), (True, 1, 1), (True, 4, 0), (True, 64, 1)])
def test_a_run_between_splices_evictions_and_frees(gqa, P, pairing):
    """Prompts, then tokens, over two layers, as a server would run them: a splice,
    an eviction and a new sequence in between; a step that no longer fits its
    sequences is refused."""
    say(f"run gqa={gqa} P={P}")
    c = Cache(gqa, P, [5 * P + 3, 40, 1], seed=P, layers=2, kv_heads=2, dim=64, rot=32, pairing=pairing, spare=-(-400 // P) + 8, room=400)
    L, heads = c.L, 6 if gqa else 5
    step = c.pool.step(heads, max_seqs=3, max_tokens=160)
    g = np.random.default_rng(P)
    plan = [([0, 1, 2], [0, 70, 33]), ([2, 0], [1, 1]), ([0, 1, 2], [1, 1, 1]), ([1, 0], [2, 3]), ([2, 1, 0], [120, 1, 1]),
            ([0, 1, 2], [1, 1, 1])]
    for i, (seqs, counts) in enumerate(plan):
        _run_step(c, step, seqs, counts, heads, g, 2)
        if i == 1:
            c.pool.splice([L.Directive(0, 2, 5)])
        elif i == 2:
            n = c.pool.seq_get(1)[0]
            keep = torch.from_numpy((g.random(n) > 0.3).astype(np.uint8)).cuda()
            c.pool.evict([1], keep, [0])
        elif i == 3:
            c.pool.seq_free(2)
            assert c.pool.seq_alloc(0) == 2
            _run_step(c, step, [0, 1], [1, 1], heads, g, 2)   # the others go on
            continue
        else:
            continue
        T = sum(counts)
        q = torch.zeros((T, heads, 64 if gqa else 576), dtype=torch.bfloat16, device="cuda")
        with pytest.raises(L.LeylineError):
            step.attend(0, q, scale=1.0)
        with pytest.raises(L.LeylineError):
            step.append(0, q=q[..., :64])
    step.close()
    c.pool.close()


@pytest.mark.parametrize("gqa", [False, True])
def test_captured_steps_replay(gqa):
    """Two layers' append and attention in one graph, replayed after begins of
    other sizes (none, one token, chunks, a growing split), with eager work and
    other steps' calls between; buffer rows behind the last token stay."""
    say(f"graph gqa={gqa}")
    c = Cache(gqa, 16, [600, 37, 16], seed=9, layers=2, kv_heads=2, dim=128, rot=128, pairing=1, spare=40, room=300)
    heads, cap = 8, 24
    step, other = c.pool.step(heads, max_seqs=3, max_tokens=cap), c.pool.step(heads, max_seqs=3, max_tokens=cap)
    dq, dv = (128, 128) if gqa else (64, 512)

    def buf(*shape):
        return torch.zeros(shape, dtype=torch.bfloat16, device="cuda")
    if gqa:
        a, b, lat = [buf(cap, 2, 128) for _ in range(2)], [buf(cap, 2, 128) for _ in range(2)], None
    else:
        a, b = [buf(cap, 512) for _ in range(2)], [buf(cap, 64) for _ in range(2)]
        lat = buf(cap, heads, 512)
    q, qo, out = buf(cap, heads, dq), [buf(cap, heads, dq) for _ in range(2)], [buf(cap, heads, dv) for _ in range(2)]
    lse = [torch.zeros((cap, heads), dtype=torch.float32, device="cuda") for _ in range(2)]
    scale = 128 ** -0.5 if gqa else 0.05

    def layers(s):
        for i in range(2):
            s.append(i, a[i], b[i], q=q, q_out=qo[i])
            if gqa:
                s.attend(i, qo[i], scale=scale, out=out[i], lse=lse[i])
            else:
                s.attend(i, lat, qo[i], scale=scale, out=out[i], lse=lse[i])
    step.begin([0], [1], grow=False)   # (a grown row that nothing has written is NaN here, and seen)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    stream = torch.cuda.Stream()
    with torch.cuda.graph(graph, stream=stream):
        with pytest.raises(c.L.LeylineError):
            step.begin([0], [1])
        with pytest.raises(c.L.LeylineError):
            step.append(0, q=q[:cap - 1])   # too little room for a later begin
        layers(step)
    g = np.random.default_rng(2)
    plans = [([0, 1], [1, 1]), ([0, 1, 2], [1, 20, 3]), ([2], [1]), ([], []), ([1, 0], [12, 12]), ([0], [1]), ([0, 2], [24, 0])]
    for seqs, counts in plans:
        for t in a + b + [q] + ([] if gqa else [lat]):
            t.copy_(bf16(g.standard_normal(tuple(t.shape))))
        for t in qo + out:
            t.fill_(7.0)
        for t in lse:
            t.fill_(7.0)
        before = {s: c.pool.seq_get(s)[:2] for s in seqs}
        torch.cuda.synchronize()
        with torch.cuda.stream(stream):
            T = step.begin(seqs, counts)
            graph.replay()
        torch.cuda.synchronize()
        for i in range(2):
            assert (f64(qo[i])[T:] == 7).all() and (f64(out[i])[T:] == 7).all() and (f64(lse[i])[T:] == 7).all()
            full = qo[i] if gqa else torch.cat([lat, qo[i]], -1)
            c.check_attend(out[i][:T], lse[i][:T], full[:T], seqs, counts, i, scale)
        if not T:
            continue
        rows = [[c.rows(p, i, s, before[s][0]) for s in seqs for p in range(len(c.planes))] for i in range(2)]
        graphed = [x.clone() for x in qo + out]
        # eager, on the same tokens, by another step: the same rows and queries bit
        # for bit, the attention within its tolerance (it may take other tiles)
        other.begin(seqs, counts, grow=False)
        layers(other)
        torch.cuda.synchronize()
        for i in range(2):
            again = [c.rows(p, i, s, before[s][0]) for s in seqs for p in range(len(c.planes))]
            assert all(np.array_equal(x, y) for x, y in zip(rows[i], again))
            assert torch.equal(qo[i], graphed[i])
            full = qo[i] if gqa else torch.cat([lat, qo[i]], -1)
            c.check_attend(out[i][:T], lse[i][:T], full[:T], seqs, counts, i, scale)
        # a replay without a begin in between does the same again
        with torch.cuda.stream(stream):
            graph.replay()
            graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(graphed, qo + out))
    for s in (step, other):
        s.close()
    c.pool.close()


@pytest.mark.parametrize("gqa", [False, True])
def test_calls_on_other_streams_follow_one_another(gqa):
    c = Cache(gqa, 16, [500, 31], seed=2, layers=1, kv_heads=1, dim=64, rot=64, spare=20, room=100)
    step = c.pool.step(4, max_tokens=8)
    g = np.random.default_rng(0)
    streams = [torch.cuda.Stream() for _ in range(3)]
    for turn in range(4):
        a = bf16(g.standard_normal((3, 1, 64) if gqa else (3, 512))).cuda()
        b = bf16(g.standard_normal((3, 1, 64) if gqa else (3, 64))).cuda()
        q = bf16(g.standard_normal((3, 4, 64 if gqa else 576))).cuda()
        before = c.pool.seq_get(0)[0]
        torch.cuda.synchronize()
        step.begin([0, 1], [1, 2], stream=streams[turn % 3])
        step.append(0, a, b, stream=streams[(turn + 1) % 3])
        with torch.cuda.stream(streams[(turn + 2) % 3]):
            out, lse = step.attend(0, q, scale=0.1, lse=True)
        torch.cuda.synchronize()
        assert c.pool.seq_get(0)[0] == before + 1
        got = c.rows(1 if gqa else 0, 0, 0, before)[0, 0, :64]
        if gqa:
            assert np.array_equal(got, f64(b)[0, 0])
        else:
            assert np.array_equal(got, f64(a)[0, :64])
        c.check_attend(out, lse, q, [0, 1], [1, 2], 0, 0.1)
    step.close()
    c.pool.close()


@pytest.mark.parametrize("gqa", [False, True])
def test_views_and_spare_rows(gqa):
    """Head-major outputs, padded and shared (stride 0) queries, a separate rotated
    part, more buffer rows than tokens: only the tokens' values are written."""
    c = Cache(gqa, 4, [90, 33], seed=8, kv_heads=2, dim=80, rot=16)
    heads, n = 6, 80 if gqa else 512
    step = c.pool.step(heads, max_tokens=40)
    T = step.begin([1, 0], [7, 20], grow=False)
    wide = _queries(c, T + 3, heads + 1)
    big = torch.full((heads, T + 5, n + 8), 7.0, dtype=torch.bfloat16, device="cuda")
    out = big[:, :, :n].transpose(0, 1)
    lse = torch.full((T + 5, heads), 7.0, dtype=torch.float32, device="cuda")
    kw = dict(scale=0.07, window=50)
    if gqa:
        step.attend(0, wide[:, 1:], out=out, lse=lse, **kw)
    else:
        pe = wide[:, 1:, 512:].contiguous()
        step.attend(0, wide[:, 1:, :512], pe, out=out, lse=lse, **kw)
    c.check_attend(out[:T], lse[:T], wide[:T, 1:], [1, 0], [7, 20], 0, 0.07, True, 50)
    assert (f64(big)[:, T:] == 7).all() and (f64(big)[..., n:] == 7).all() and (f64(lse)[T:] == 7).all()
    one = wide[:, :1].expand(-1, heads, -1)   # every head the same query
    got, l = step.attend(0, one, lse=True, scale=0.07)
    c.check_attend(got[:T], l[:T], one[:T].contiguous(), [1, 0], [7, 20], 0, 0.07)
    with pytest.raises(c.L.LeylineError):   # rows of the result on top of each other
        step.attend(0, wide[:, 1:], out=torch.zeros((T, 1, n), dtype=torch.bfloat16, device="cuda").expand(-1, heads, -1), **kw)
    with pytest.raises(c.L.LeylineError):   # too few of them
        step.attend(0, wide[:T - 1, 1:], **kw)
    with pytest.raises(c.L.LeylineError):   # not 16-byte aligned
        step.attend(0, torch.zeros((T, heads, (n if gqa else 576) + 8), dtype=torch.bfloat16, device="cuda")[..., 4:-4], **kw)
    step.close()
    c.pool.close()


@pytest.mark.parametrize("gqa", [False, True])
def test_offsets_past_32_bits(gqa):
    """Cache rows more than 2^32 values into their plane, and query tokens 2^32
    values apart."""
    L = need_gpu()
    row, P, n = (1024, 256, 700) if gqa else (576, 256, 700)
    pages = ((1 << 32) + (1 << 24)) // (row * P)
    shape = (1, pages, P, 8, 128) if gqa else (1, pages, P, 576)
    planes = [torch.empty(shape, dtype=torch.bfloat16, device="cuda") for _ in range(2 if gqa else 1)]
    table = torch.full((1, 4), -1, dtype=torch.int32, device="cuda")
    c = object.__new__(Cache)
    c.L, c.gqa, c.P, c.layers, c.H, c.D, c.rot, c.pairing, c.base = L, gqa, P, 1, 8, 128, 128, 1, 10000.0
    c.planes = planes
    c.pool = L.GqaPool(planes[0], planes[1], table, pairing=1) if gqa else L.Pool(planes[0], table, pairing=1)
    c.pool.seq_set_pages(0, [pages - 1, 3, pages - 2], n)
    g = np.random.default_rng(3)
    for x in planes:
        x.view(-1, *shape[3:])[c.slots(0, 0, n)] = bf16(g.standard_normal((n, *shape[3:]))).cuda()
    heads = 8
    step = c.pool.step(heads, max_tokens=2)
    dq = 128 if gqa else 576
    far = (1 << 32) - 64
    store = torch.empty(far + heads * dq, dtype=torch.bfloat16, device="cuda")
    q = store.as_strided((2, heads, dq), (far, dq, 1))
    q.copy_(bf16(g.standard_normal((2, heads, dq))).cuda())
    before = c.pool.seq_get(0)[:2]
    step.begin([0], [2])
    a = bf16(g.standard_normal((2, 8, 128) if gqa else (2, 512))).cuda()
    b = bf16(g.standard_normal((2, 8, 128) if gqa else (2, 64))).cuda()
    step.append(0, a, b, q=q[..., -dq if gqa else -64:], q_out=q[..., -dq if gqa else -64:])
    out, lse = step.attend(0, q, scale=0.05, lse=True)
    torch.cuda.synchronize()
    ang = S.angles(before[1] + np.arange(2), 128 if gqa else 64, 10000.0)
    if gqa:
        c.check_rows(0, 0, 0, n, n + 2, *S.heads(f64(a), None, 0, ang, 1, 128))
        assert np.array_equal(c.rows(1, 0, 0, n, n + 2), f64(b))
    else:
        assert np.array_equal(c.rows(0, 0, 0, n, n + 2)[:, 0, :512], f64(a))
    c.check_attend(out, lse, q.contiguous(), [0], [2], 0, 0.05)
    step.close()
    c.pool.close()


@pytest.mark.parametrize("gqa", [False, True])
def test_overwritten_page_tables_stay_inside_the_pool(gqa):
    """Page numbers that no pool call wrote: attention reads page 0 for them,
    append writes no row, other sequences and pages are not touched."""
    c = Cache(gqa, 16, [100, 60], seed=7, kv_heads=2, dim=64)
    step = c.pool.step(4, max_tokens=8)
    keep = c.table.clone()
    c.table[0, :] = c.planes[0].shape[1]   # one past the last page
    c.table[0, 1::2] = -(1 << 31)
    c.table[0, 2::4] = (1 << 31) - 1
    step.begin([0, 1], [3, 2], grow=False)
    q = _queries(c, 5, 4)
    before = [x.clone() for x in c.planes]
    a = torch.ones((5, 2, 64) if gqa else (5, 512), dtype=torch.bfloat16, device="cuda")
    b = torch.ones((5, 2, 64) if gqa else (5, 64), dtype=torch.bfloat16, device="cuda")
    step.append(0, a, b)
    out = step.attend(0, q, scale=0.1)
    torch.cuda.synchronize()
    rows = c.slots(1, 58, 60)
    for x, y in zip(c.planes, before):
        x, y = x.view(-1, *x.shape[3:]), y.view(-1, *y.shape[3:])
        untouched = torch.ones(x.shape[0], dtype=torch.bool, device="cuda")
        untouched[rows] = False
        assert torch.equal(x[untouched].view(torch.int16), y[untouched].view(torch.int16))
        assert not torch.equal(x[rows].view(torch.int16), y[rows].view(torch.int16))
    c.check_attend(out[3:], None, q[3:], [1], [2], 0, 0.1)
    c.table.copy_(keep)
    step.begin([0], [3], grow=False)
    out = step.attend(0, q[:3], scale=0.1)
    c.check_attend(out, None, q[:3], [0], [3], 0, 0.1)
    step.close()
    c.pool.close()


@pytest.mark.parametrize("gqa", [False, True])
def test_empty_steps_and_refused_begins(gqa):
    """No sequences, sequences without tokens, sequences without rows; begins that
    are refused leave the step and the pool as they were."""
    c = Cache(gqa, 16, [20, 0, 5], seed=1, kv_heads=1, dim=64, spare=1)
    E = c.L.LeylineError
    step, d = c.pool.step(2, max_seqs=2, max_tokens=9), 64 if gqa else 576
    q = _queries(c, 9, 2)
    with pytest.raises(E):
        step.attend(0, q, scale=0.1)   # not begun
    for seqs, counts in (([], []), ([1, 0], [0, 0])):
        assert step.begin(seqs, counts) == 0
        assert step.attend(0, q[:0], scale=0.1).shape == (0, 2, 64 if gqa else 512)
        out = torch.full((4, 2, 64 if gqa else 512), 7.0, dtype=torch.bfloat16, device="cuda")
        step.attend(0, q[:4], scale=0.1, out=out)
        assert (out == 7).all()
        assert step.append(0, q=q[:0, :, :64]).shape == (0, 2, 64)
    assert step.begin([0, 2], [3, 5], grow=False) == 8
    want = step.attend(0, q, scale=0.1)
    books = [c.pool.seq_get(i)[:2] for i in range(3)]
    for seqs, counts, grow in (([0, 0], [1, 1], True), ([0, 3], [1, 1], True), ([0], [-1], True), ([0, 1, 2], [1, 1, 1], True),
                               ([0], [10], True), ([1], [1], False), ([0, 2], [8, 9], True), ([0, -1], [1, 1], True)):
        with pytest.raises(E):
            step.begin(seqs, counts, grow=grow)
    assert books == [c.pool.seq_get(i)[:2] for i in range(3)]
    again = step.attend(0, q, scale=0.1)   # the step begun last still stands
    assert torch.equal(want[:8], again[:8])
    c.check_attend(again[:8], None, q[:8], [0, 2], [3, 5], 0, 0.1)
    c.pool.close()
    with pytest.raises(E):
        step.attend(0, q, scale=0.1)
    with pytest.raises(E):
        step.begin([0], [1])
    step.close()


def test_pools_of_2_to_the_31_rows_a_sequence_are_refused():
    L = need_gpu()
    k = torch.zeros((1, 2, 256, 1, 16), dtype=torch.bfloat16, device="cuda")
    for width, ok in ((((1 << 31) - 1024) // 256, False), (((1 << 31) - 1024) // 256 - 1, True)):
        pool = L.GqaPool(k, k.clone(), torch.full((1, width), -1, dtype=torch.int32, device="cuda"), rotary_dim=16)
        if ok:
            pool.step(2, max_tokens=1).close()
        else:
            with pytest.raises(L.LeylineError, match="2\\^31"):
                pool.step(2, max_tokens=1)
        pool.close()


@pytest.mark.parametrize("gqa,heads,kv,dim,rot,pairing,norm", [
    (False, 43, 1, 576, 64, 0, True), (False, 40, 1, 576, 64, 1, False),
    (True, 15, 3, 96, 32, 0, True), (True, 14, 7, 64, 64, 1, True), (True, 9, 3, 256, 64, 1, False),
])
def test_append_of_many_tokens(gqa, heads, kv, dim, rot, pairing, norm):
    """Prompts of odd lengths, enough heads and tokens for more than one round of
    the chip's waves (the kernel's other form); one call of rows or queries alone."""
    say(f"many tokens gqa={gqa} heads={heads}/{kv} dim={dim} pairing={pairing} norm={norm}")
    lens, counts = [5, 0, 77], [1501, 800, 0]
    c = Cache(gqa, 16, lens, seed=3, kv_heads=kv, dim=dim, rot=rot, pairing=pairing, room=1600, spare=150)
    step = c.pool.step(heads, max_tokens=2400)
    T = step.begin([0, 1, 2], counts)
    g = np.random.default_rng(5)
    dq = dim if gqa else 64
    a = bf16(g.standard_normal((T, kv, dim) if gqa else (T, 512))).cuda()
    b = bf16(g.standard_normal((T, kv, dim) if gqa else (T, 64))).cuda()
    wide = bf16(g.standard_normal((T, heads, dq + 8))).cuda()
    q = wide[..., 8:]
    w = bf16(g.standard_normal(dim if gqa else 512)).cuda() if norm else None
    qw = bf16(g.standard_normal(dim)).cuda() if norm and gqa else None
    out = torch.full((T + 2, heads, dq + 8), 7.0, dtype=torch.bfloat16, device="cuda")
    step.append(0, a, b, norm=w, q=q, q_out=out[:, :, :dq], q_norm=qw, eps=1e-5)
    torch.cuda.synchronize()
    ang = S.angles(np.concatenate([lens[i] + np.arange(counts[i]) for i in (0, 1)]), rot, 10000.0)
    ww, qww = (None if x is None else f64(x) for x in (w, qw))
    want, size = S.heads(f64(q), qww, 1e-5, ang, pairing, rot)
    got = f64(out)
    assert (np.abs(got[:T, :, :dq] - want) <= HALF_STEP * np.abs(want) + 2.0 ** -18 * size).all()
    assert (got[T:] == 7).all() and (got[..., dq:] == 7).all()
    lo = 0
    for i in (0, 1):
        sl, at = slice(lo, lo + counts[i]), (i, lens[i], lens[i] + counts[i])
        if gqa:
            c.check_rows(0, 0, *at, *S.heads(f64(a[sl]), ww, 1e-5, ang[sl], pairing, rot))
            assert np.array_equal(c.rows(1, 0, *at), f64(b[sl]))
        else:
            lat = S.norm(f64(a[sl])[:, None], ww, 1e-5)
            pe, sp = S.heads(f64(b[sl])[:, None], None, 0, ang[sl], pairing)
            c.check_rows(0, 0, *at, np.concatenate([lat, pe], -1), np.concatenate([np.abs(lat), sp], -1))
        lo += counts[i]
    rows = [c.rows(p, 0, 0) for p in range(len(c.planes))]
    again = step.append(0, q=q, q_norm=qw, eps=1e-5)
    assert torch.equal(again, out[:T, :, :dq])
    step.append(0, a, b, norm=w, eps=1e-5)
    assert all(np.array_equal(x, c.rows(p, 0, 0)) for p, x in enumerate(rows))
    step.close()
    c.pool.close()
