"""The serving step at the limits of what it promises, on the GPU: tokens whose
scores are all -inf, far positions, steps that run eagerly after a capture,
begins behind an eviction that need no page.  Tolerances are those of
test_gpu_step.py."""

import numpy as np
import pytest

from oracle import step_oracle as S

from gpu_common import say, torch
from test_gpu_step import F32, HALF_STEP, Cache, _cache, _queries, bf16, f64

pytestmark = pytest.mark.gpu

INF = float("inf")


@pytest.mark.parametrize("kind", ["mla", "gqa64", "gqa128", "gqa256"])
@pytest.mark.parametrize("count", [1, 3, 7, 15, 33])
@pytest.mark.parametrize("n", [64, 1280])
@pytest.mark.parametrize("causal", [True, False])
def test_scores_that_are_all_minus_infinity(kind, count, n, causal):
    """Every key is -inf where the queries are 1, and so is a column of every value
    (MLA: the same one; GQA: +inf): zeros and lse = -inf, in every tile (8 to 264
    query rows), whole (64 rows) and split, read in tiles and row by row."""
    say(f"all -inf {kind} count={count} n={n} causal={causal}")
    gqa, dim = kind != "mla", int(kind[3:] or 0) if kind != "mla" else 576
    c = _cache(gqa, 1, dim, 16, [n], seed=3)
    s = c.slots(0, 0, n)
    for plane, value in zip(c.planes, (-INF, INF)):
        x = plane[0].view(-1, *plane.shape[3:])
        x[s, ..., 5] = value
    heads = 8
    q = torch.zeros((count, heads, dim), dtype=torch.bfloat16, device="cuda")
    q[..., 5] = 1.0
    step = c.pool.step(heads, max_tokens=count)
    step.begin([0], [count], grow=False)
    out, lse = step.attend(0, q, scale=0.1, causal=causal, lse=True)
    torch.cuda.synchronize()
    assert (f64(out) == 0).all() and (f64(lse) == -INF).all()
    step.close()
    c.pool.close()


@pytest.mark.parametrize("gqa", [False, True])
@pytest.mark.parametrize("P", [1, 16])
def test_begins_behind_an_eviction_that_need_no_page(gqa, P):
    """The host's page list stays out of date until a begin needs it: the last rows
    asked again, a row in a page that is there, then rows in new pages."""
    c = Cache(gqa, P, [300], seed=P, kv_heads=2, dim=64, rot=64, room=80, spare=-(-380 // P) + 4)
    step = c.pool.step(4, max_tokens=40)
    g = np.random.default_rng(8)
    keep = (g.random(300) > 0.4).astype(np.uint8)
    while P > 1 and keep.sum() % P != P // 2:
        keep[np.flatnonzero(keep)[0]] = 0
    want = [c.rows(p, 0, 0)[keep == 1] for p in range(len(c.planes))]
    n = int(keep.sum())
    c.pool.evict([0], torch.from_numpy(keep).cuda(), [0])
    outs = []
    for count, grow in ((3, False), (1, True), (40, True)):
        T = step.begin([0], [count], grow=grow)
        q = _queries(c, T, 4, seed=count)
        if grow:
            a = bf16(g.standard_normal((T, 2, 64) if gqa else (T, 512))).cuda()
            b = bf16(g.standard_normal((T, 2, 64) if gqa else (T, 64))).cuda()
            step.append(0, a, b)
        outs.append((count, q, *step.attend(0, q, scale=0.1, lse=True)))
    torch.cuda.synchronize()
    assert c.pool.seq_get(0)[:2] == (n + 41, 341)
    for p in range(len(c.planes)):
        assert np.array_equal(c.rows(p, 0, 0, 0, n), want[p])
    count, q, out, lse = outs[-1]
    c.check_attend(out, lse, q, [0], [count], 0, 0.1)
    # the first two, against the rows that were there then
    for (count, q, out, lse), rows in zip(outs, (n, n + 1)):
        k = c.rows(0, 0, 0, 0, rows)
        v = c.rows(1, 0, 0, 0, rows) if gqa else k[..., :512]
        for h in range(4):
            x = h // (4 // k.shape[1])
            o, l, w, slack = S.attend(f64(q)[:, h], k[:, x], v[:, x], rows - count, 0.1)
            ds = k.shape[-1] * F32 * slack[:, None] + 8 * F32 * (1 + np.abs(l[:, None]))
            assert (np.abs(f64(out)[:, h] - o) <= HALF_STEP * (np.abs(o) + w) + (2 * ds + rows * F32) * w + 1e-30).all()
            assert (np.abs(f64(lse)[:, h] - l) <= ds[:, 0] + rows * F32).all()
    step.close()
    c.pool.close()


@pytest.mark.parametrize("gqa,pairing", [(False, 0), (False, 1), (True, 0), (True, 1)])
def test_append_at_a_far_position(gqa, pairing):
    """An eviction keeps positions: of 2^20 + 77 rows 40 stay, and the next tokens
    are rows 40 on at positions 2^20 + 77 on."""
    n, held, T, heads = (1 << 20) + 77, 40, 5, 6
    c = Cache(gqa, 256, [0], kv_heads=1, dim=32, rot=32, pairing=pairing, base=500000.0, room=n + 512, spare=n // 256 + 2)
    c.pool.seq_set_pages(0, list(range(-(-n // 256))), n)
    keep = torch.zeros(n, dtype=torch.uint8, device="cuda")
    keep[torch.arange(held, device="cuda") * 25000] = 1
    c.pool.evict([0], keep, [0])
    step = c.pool.step(heads, max_tokens=T)
    assert step.begin([0], [T]) == T
    assert c.pool.seq_get(0)[:2] == (held + T, n + T)
    g = np.random.default_rng(1)
    ang = S.angles(n + np.arange(T), 32 if gqa else 64, 500000.0)
    a, b = (bf16(g.standard_normal((T, 1, 32) if gqa else (T, w))).cuda() for w in (512, 64))
    q = bf16(g.standard_normal((T, heads, 32 if gqa else 64))).cuda()
    qo = step.append(0, a, b, q=q)
    torch.cuda.synchronize()
    if gqa:
        c.check_rows(0, 0, 0, held, held + T, *S.heads(f64(a), None, 0, ang, pairing, 32))
        assert np.array_equal(c.rows(1, 0, 0, held, held + T), f64(b))
    else:
        pe, size = S.heads(f64(b)[:, None], None, 0, ang, pairing)
        lat = f64(a)[:, None]
        c.check_rows(0, 0, 0, held, held + T, np.concatenate([lat, pe], -1), np.concatenate([np.abs(lat), size], -1))
    want, size = S.heads(f64(q), None, 0, ang, pairing)
    assert (np.abs(f64(qo) - want) <= HALF_STEP * np.abs(want) + 2.0 ** -18 * size).all()
    step.close()
    c.pool.close()


@pytest.mark.parametrize("gqa", [False, True])
@pytest.mark.parametrize("captured,eager", [(1, 70), (70, 1)])
def test_eager_calls_beside_a_graph(gqa, captured, eager):
    """A step whose attention a graph holds: its eager calls give the bits of a step
    that no graph holds, the graph's replays go on, in turn and behind each other."""
    say(f"eager beside a graph gqa={gqa} captured={captured} eager={eager}")
    c = Cache(gqa, 16, [900, 333], seed=11, kv_heads=2, dim=128, rot=128)
    heads, cap = 8, 80
    step, other = (c.pool.step(heads, max_seqs=2, max_tokens=cap) for _ in range(2))
    q, dv = _queries(c, cap, heads), 128 if gqa else 512
    out = torch.zeros((cap, heads, dv), dtype=torch.bfloat16, device="cuda")
    lse = torch.zeros((cap, heads), dtype=torch.float32, device="cuda")

    def both(s, count):
        T = s.begin([1, 0], [count, count // 7], grow=False)
        return T, s.attend(0, q, scale=0.09, lse=True)
    _, want = both(other, eager)   # (also loads the kernels)
    step.begin([1, 0], [captured, captured // 7], grow=False)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    stream = torch.cuda.Stream()
    with torch.cuda.graph(graph, stream=stream):
        step.attend(0, q, scale=0.09, out=out, lse=lse)
    for turn in range(3):
        T, got = both(step, eager)
        torch.cuda.synchronize()
        assert torch.equal(got[0][:T].view(torch.int16), want[0][:T].view(torch.int16))
        assert torch.equal(got[1][:T], want[1][:T])
        for count in (captured, eager):   # replays of the size captured, and of the other
            out.fill_(7.0)
            torch.cuda.synchronize()
            with torch.cuda.stream(stream):
                T = step.begin([1, 0], [count, count // 7], grow=False)
                graph.replay()
                graph.replay()
            torch.cuda.synchronize()
            c.check_attend(out[:T], lse[:T], q[:T], [1, 0], [count, count // 7], 0, 0.09)
            assert (out[T:] == 7).all()
    for s in (step, other):
        s.close()
    c.pool.close()
