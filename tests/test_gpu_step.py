"""GPU parity of the serving step (append and attend of include/leyline_step.h)
against the float64 oracle, through the binding: MLA and GQA pools, one token to
chunks, odd sizes, views, masks, several layers, steps between splices and
evictions.  Every row of the pool that no sequence holds is NaN, so that a read
past a sequence's end shows.

Tolerances.  append: the result is rounded once (bf16, half a step: 2^-8 of the
value); the float32 work before it is a sum of n squares (a norm) and two
products, each off by 2^-24 of its terms: 2^-18 of the magnitudes that enter.
attend: the softmax weights are rounded to bf16 (2^-8 of each, so 2^-8 of
sum p |v|) and the result once more (2^-8); a score is a float32 sum of dk
products, off by at most dk 2^-24 sum |q k|, which shifts every weight and the
sum of weights by that much relatively; the float32 sums over n rows add n 2^-24."""

import numpy as np
import pytest

from oracle import step_oracle as S
from synth import permuted_pages

from gpu_common import need_gpu, say, torch

pytestmark = pytest.mark.gpu

HALF_STEP = 2.0 ** -8
F32 = 2.0 ** -24


def bf16(x):
    return torch.from_numpy(np.ascontiguousarray(x, np.float32)).to(torch.bfloat16)


def f64(t):
    return t.detach().float().cpu().numpy().astype(np.float64)


class Cache:
    """A pool with sequences on permuted pages, random live rows, NaN elsewhere."""

    def __init__(self, gqa, P, lens, seed=0, layers=1, kv_heads=2, dim=64, rot=64, pairing=0, base=10000.0, spare=8,
                 room=0):
        L = need_gpu()
        self.L, self.gqa, self.P, self.layers = L, gqa, P, layers
        self.H, self.D, self.rot, self.pairing, self.base = kv_heads, dim, rot, pairing, base
        self.rng = np.random.default_rng(seed)
        per = [-(-n // P) for n in lens]
        pages = sum(per) + spare
        self.lens = list(lens)
        self.width = max(per + [1]) + -(-room // P) + 1
        self.table = torch.full((len(lens), self.width), -1, dtype=torch.int32, device="cuda")
        shape = (layers, pages, P, kv_heads, dim) if gqa else (layers, pages, P, 576)
        self.planes = [torch.full(shape, float("nan"), dtype=torch.bfloat16, device="cuda") for _ in range(2 if gqa else 1)]
        if gqa:
            self.pool = L.GqaPool(self.planes[0], self.planes[1], self.table, rotary_dim=rot, pairing=pairing, rope_base=base)
        else:
            self.pool = L.Pool(self.planes[0], self.table, pairing=pairing, rope_base=base)
        order = permuted_pages(seed, pages)
        at = 0
        for i, n in enumerate(lens):
            self.pool.seq_set_pages(i, order[at:at + per[i]], n)
            at += per[i]
            slots = self.slots(i, 0, n)
            for x in self.planes:
                rows = x.view(layers, -1, *shape[3:])
                rows[:, slots] = bf16(self.rng.standard_normal((layers, n, *shape[3:]))).cuda()

    def slots(self, seq, lo, hi):
        pages = self.pool.seq_get(seq)[2].astype(np.int64)
        j = np.arange(lo, hi)
        return torch.from_numpy(pages[j // self.P] * self.P + j % self.P).cuda()

    def rows(self, plane, layer, seq, lo=0, hi=None):
        """Rows of a sequence as float64 [n][heads][dim] (MLA: [n][1][576])."""
        hi = self.pool.seq_get(seq)[0] if hi is None else hi
        x = self.planes[plane][layer]
        x = x.view(-1, *x.shape[2:])[self.slots(seq, lo, hi)]
        return f64(x if self.gqa else x[:, None])

    def check_attend(self, out, lse, q, seqs, counts, layer, scale, causal=True, window=0, first=None):
        """out / lse [T][heads][*] against the oracle on the cache as it is; returns
        the worst error over its tolerance."""
        T, heads, _ = q.shape
        got, ql = f64(out), f64(q)
        gl = None if lse is None else f64(lse)
        worst, at = 0.0, 0
        for i, (s, n) in enumerate(zip(seqs, counts)):
            k = self.rows(0, layer, s)
            v = self.rows(1, layer, s) if self.gqa else k[..., :512]
            f = k.shape[0] - n if first is None else first[i]
            for h in range(heads):
                kv = h // (heads // k.shape[1])
                o, l, w, slack = S.attend(ql[at:at + n, h], k[:, kv], v[:, kv], f, scale, causal, window)
                ds = k.shape[-1] * F32 * slack[:, None] + 8 * F32 * (1 + np.abs(l[:, None]))
                tol = HALF_STEP * (np.abs(o) + w) + (2 * ds + k.shape[0] * F32) * w + 1e-30
                bad = np.abs(got[at:at + n, h] - o) / tol
                assert np.isfinite(bad).all(), (s, h, np.argwhere(~np.isfinite(bad))[:4].tolist())
                worst = max(worst, float(bad.max(initial=0.0)))
                assert worst <= 1, (s, h, worst, np.argwhere(bad > 1)[:4].tolist())
                if gl is not None:
                    e = np.abs(gl[at:at + n, h] - l) / (ds[:, 0] + k.shape[0] * F32 + 1e-30)
                    assert (e <= 1).all(), (s, h, float(e.max()))
            at += n
        return worst

    def check_rows(self, plane, layer, seq, lo, hi, want, size):
        got = self.rows(plane, layer, seq, lo, hi)
        tol = HALF_STEP * np.abs(want) + 2.0 ** -18 * size + 1e-30
        assert (np.abs(got - want) <= tol).all(), (seq, float((np.abs(got - want) / tol).max()))


ATTEND = [
    # gqa, heads, kv_heads, dim, page, lengths, counts
    (False, 16, 1, 576, 16, [1], [1]),
    (False, 16, 1, 576, 16, [700], [1]),
    (False, 16, 1, 576, 1, [65, 3, 130], [1, 1, 1]),
    (False, 1, 1, 576, 4, [77, 1], [1, 1]),
    (False, 20, 1, 576, 64, [200, 333], [1, 2]),
    (False, 8, 1, 576, 256, [300], [37]),
    (False, 128, 1, 576, 16, [129, 64], [1, 2]),
    (False, 16, 1, 576, 16, [150, 40, 0, 16], [150, 0, 0, 5]),
    (False, 40, 1, 576, 16, [97], [2]),
    (True, 4, 2, 64, 16, [1, 500], [1, 1]),
    (True, 8, 2, 128, 16, [700, 33], [1, 1]),
    (True, 15, 3, 96, 4, [130, 77, 5], [30, 1, 5]),
    (True, 8, 8, 32, 1, [70], [9]),
    (True, 5, 1, 80, 16, [260], [100]),
    (True, 6, 2, 256, 64, [190, 65], [65, 1]),
    (True, 2, 1, 8, 16, [50], [50]),
    (True, 64, 1, 128, 16, [100, 31], [3, 31]),
]


def _queries(c, T, heads, seed=5):
    g = np.random.default_rng(seed)
    return bf16(g.standard_normal((T, heads, c.D if c.gqa else 576))).cuda()


def _rot(dim):
    r = 16
    while r * 2 <= dim and dim % (r * 2) == 0:
        r *= 2
    return r


def _cache(gqa, kv_heads, dim, P, lens, **kw):
    # a band of 16 has to divide the head; heads narrower than that go with head 16
    return Cache(gqa, P, lens, kv_heads=kv_heads, dim=dim, rot=_rot(dim), **kw) if gqa else Cache(False, P, lens, **kw)


@pytest.mark.parametrize("gqa,heads,kv_heads,dim,P,lens,counts", ATTEND)
@pytest.mark.parametrize("mask", ["causal", "window", "all"])
def test_attend_matches_the_oracle(gqa, heads, kv_heads, dim, P, lens, counts, mask):
    say(f"attend gqa={gqa} heads={heads}/{kv_heads} dim={dim} P={P} lens={lens} counts={counts} {mask}")
    if gqa and dim < 16:
        dim = 16
    c = _cache(gqa, kv_heads, dim, P, lens, seed=heads + P)
    step = c.pool.step(heads, max_tokens=max(1, sum(counts)))
    seqs = list(range(len(lens)))
    T = step.begin(seqs, counts, grow=False)
    q = _queries(c, T, heads)
    scale = 0.07 if not gqa else dim ** -0.5
    kw = dict(causal=mask != "all", window=29 if mask == "window" else 0)
    out, lse = step.attend(0, q, scale=scale, lse=True, **kw)
    again, lse2 = step.attend(0, q, scale=scale, lse=True, **kw)
    torch.cuda.synchronize()
    worst = c.check_attend(out, lse, q, seqs, counts, 0, scale, kw["causal"], kw["window"])
    assert torch.equal(out.view(torch.int16), again.view(torch.int16)) and torch.equal(lse, lse2)
    say(f"  worst error / tolerance {worst:.3f}")
    step.close()
    c.pool.close()


APPEND = [
    # gqa, heads, kv_heads, dim, rot, pairing, page
    (False, 16, 1, 576, 64, 0, 16),
    (False, 5, 1, 576, 64, 1, 4),
    (False, 128, 1, 576, 64, 0, 64),
    (True, 8, 2, 128, 128, 1, 16),
    (True, 15, 3, 96, 32, 0, 4),
    (True, 4, 4, 80, 16, 1, 1),
    (True, 2, 1, 256, 64, 0, 16),
    (True, 9, 3, 16, 16, 1, 16),
]


@pytest.mark.parametrize("gqa,heads,kv_heads,dim,rot,pairing,P", APPEND)
@pytest.mark.parametrize("weights", [None, "bf16", "f32"])
def test_append_writes_rows_and_queries(gqa, heads, kv_heads, dim, rot, pairing, P, weights):
    """Growing sequences (an empty one, one that fills a page, one at a far
    position), inputs that are views of one wide projection, two layers."""
    say(f"append gqa={gqa} heads={heads}/{kv_heads} dim={dim} rot={rot} pairing={pairing} P={P} norm={weights}")
    lens, counts = [0, 2 * P, 37, 3], [P + 1, P, 1, 0]
    c = Cache(gqa, P, lens, seed=heads, layers=2, kv_heads=kv_heads, dim=dim, rot=rot, pairing=pairing, base=500000.0,
              room=2 * P, spare=8 + 3)
    L = c.L
    # a far position: rows spliced out and back leave it where it was, so use a
    # long splice of stub rows and a cut back
    before = [x.clone() for x in c.planes]
    step = c.pool.step(heads, max_seqs=4, max_tokens=64 + 2 * P)
    pos = [c.pool.seq_get(i)[1] for i in range(4)]
    T = step.begin([2, 0, 1, 3], [counts[i] for i in (2, 0, 1, 3)])
    order = [2, 0, 1]
    positions = np.concatenate([pos[i] + np.arange(counts[i]) for i in order])
    for i in range(4):
        n, p, pages = c.pool.seq_get(i)
        assert (n, p) == (lens[i] + counts[i], pos[i] + counts[i])
        assert np.array_equal(c.table[i, :len(pages)].cpu().numpy(), pages)
    dq = dim if gqa else 64
    ang = S.angles(positions, rot, 500000.0)
    g = np.random.default_rng(9)
    for layer in range(2):
        wide = bf16(g.standard_normal((T, heads * dq + 2 * kv_heads * (dim if gqa else 0) + 576 + 8))).cuda()
        q = wide[:, :heads * dq].unflatten(1, (heads, dq))
        rest = wide[:, heads * dq:]
        if gqa:
            a = rest[:, :kv_heads * dim].unflatten(1, (kv_heads, dim))
            b = rest[:, kv_heads * dim:2 * kv_heads * dim].unflatten(1, (kv_heads, dim))
        else:
            a, b = rest[:, :512], rest[:, 512:576]
        w = qw = None
        if weights:
            dt = torch.bfloat16 if weights == "bf16" else torch.float32
            w = torch.from_numpy(g.standard_normal(dim if gqa else 512)).to(dt).cuda()
            qw = torch.from_numpy(g.standard_normal(dim)).to(dt).cuda() if gqa else None
        q_out = torch.full((T + 3, heads, dq + 16), 7.0, dtype=torch.bfloat16, device="cuda")
        step.append(layer, a, b, norm=w, q=q, q_out=q_out[:, :, 8:8 + dq], q_norm=qw, eps=1e-5)
        torch.cuda.synchronize()
        lo = 0
        ww, qww = (None if w is None else f64(w)), (None if qw is None else f64(qw))
        want_q, size_q = S.heads(f64(q), qww, 1e-5, ang, pairing, rot if gqa else 64)
        got = f64(q_out)
        assert (np.abs(got[:T, :, 8:8 + dq] - want_q) <= HALF_STEP * np.abs(want_q) + 2.0 ** -18 * size_q).all()
        assert (got[T:] == 7).all() and (got[:, :, :8] == 7).all() and (got[:, :, 8 + dq:] == 7).all()
        for i in order:
            n = counts[i]
            sl = slice(lo, lo + n)
            if gqa:
                wk, sk = S.heads(f64(a[sl]), ww, 1e-5, ang[sl], pairing, rot)
                c.check_rows(0, layer, i, lens[i], lens[i] + n, wk, sk)
                assert np.array_equal(c.rows(1, layer, i, lens[i], lens[i] + n), f64(b[sl]))
            else:
                lat = S.norm(f64(a[sl])[:, None], ww, 1e-5)
                pe, sp = S.heads(f64(b[sl])[:, None], None, 0, ang[sl], pairing)
                c.check_rows(0, layer, i, lens[i], lens[i] + n, np.concatenate([lat, pe], -1),
                             np.concatenate([np.abs(lat), sp], -1))
            lo += n
    # nothing else in the pool changed
    touched = torch.cat([c.slots(i, lens[i], lens[i] + counts[i]) for i in range(4)])
    for x, y in zip(c.planes, before):
        x, y = x.view(2, -1, *x.shape[3:]), y.view(2, -1, *y.shape[3:])
        keep = torch.ones(x.shape[1], dtype=torch.bool, device="cuda")
        keep[touched] = False
        assert torch.equal(x[:, keep].view(torch.int16), y[:, keep].view(torch.int16))
    step.close()
    c.pool.close()
