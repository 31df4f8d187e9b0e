"""The operators of eviction by attention weight as they are used: rollouts served token
by token under capped scores, each token's attention added to its sequence's weights, the
heaviest rows kept every few tokens, the masks logged; then the trainer's attention over
the whole rollouts, under the death times of those logs, gives each token what serving
gave it, and its gradients are those of the same attention in float64.

Tolerance: both sides round weights and results to bf16 (2^-8 each of the value and of
sum p |v|): twice 2 * 2^-8 of the largest value."""

from dataclasses import dataclass

import numpy as np
import pytest

from oracle import weight_oracle as W

from gpu_common import need_gpu, torch

pytestmark = pytest.mark.gpu


@dataclass
class Event:
    time: int
    keep: np.ndarray


@pytest.mark.parametrize("P", [1, 16])
@pytest.mark.parametrize("dim,cap", [(64, 6.0), (96, 0.0)])
def test_serving_with_eviction_is_the_trainer_under_its_death_times(P, dim, cap):
    L = need_gpu()
    g = torch.Generator(device="cuda").manual_seed(P + dim)
    lens, prompt, Hk, G = [90, 61], 24, 2, 3
    n, T, heads = len(lens), max(lens), Hk * G

    def randn(*shape):
        return torch.randn(shape, generator=g, device="cuda").bfloat16()

    q, k, v = randn(n, T, heads, dim) * 2, randn(n, T, Hk, dim), randn(n, T, Hk, dim)
    planes = [torch.full((1, 40 if P == 16 else 400, P, Hk, dim), float("nan"), dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    rows = 128
    pool = L.GqaPool(*planes, torch.full((n, rows // P), -1, dtype=torch.int32, device="cuda"), rotary_dim=32)
    step = pool.step(heads, max_tokens=2 * prompt)
    served = torch.zeros(n, T, heads, dim, dtype=torch.bfloat16, device="cuda")
    weights = torch.zeros(n, rows, device="cuda")
    held = [[] for _ in lens]          # which token each row is
    logs = [[] for _ in lens]
    rotated = [torch.zeros(n, T, Hk, dim, dtype=torch.bfloat16, device="cuda"), torch.zeros_like(q)]
    for i in range(n):
        assert pool.seq_alloc(0) == i
    t = 0
    while t < T:
        count = prompt if t == 0 else 1
        seqs = [i for i in range(n) if t < lens[i]]
        step.begin(seqs, [count] * len(seqs))
        take = lambda x: torch.cat([x[i, t:t + count] for i in seqs])   # noqa: E731
        qt = step.append(0, take(k), take(v), q=take(q))
        out, lse = step.attend(0, qt, lse=True, cap=cap)
        step.weigh(0, qt, lse, weights, cap=cap)
        for j, i in enumerate(seqs):
            served[i, t:t + count] = out[j * count:(j + 1) * count]
            rotated[1][i, t:t + count] = qt[j * count:(j + 1) * count]
            held[i] += range(t, t + count)
            pages = pool.seq_get(i)[2].astype(np.int64)
            r = np.arange(len(held[i]) - count, len(held[i]))
            rotated[0][i, t:t + count] = planes[0][0].view(-1, Hk, dim)[torch.from_numpy(pages[r // P] * P + r % P).cuda()]
        t += count
        if t % 12 == 0:
            live = [i for i in range(n) if t < lens[i]]
            if not live:
                break
            before = [pool.seq_get(i)[0] for i in live]
            old = weights.clone()
            keep, off = pool.keep_heaviest(live, [20, 17][:len(live)], weights, sinks=2, recent=5, kept_weights=weights)
            pool.evict(live, keep, off)
            masks = keep.cpu().numpy()
            for j, i in enumerate(live):
                mask = masks[off[j]:off[j] + before[j]]
                w = old[i, :before[j]].cpu().numpy()
                assert np.array_equal(mask, W.keep_heaviest(w, [20, 17][j], 2, 5))
                logs[i].append(Event(t, mask))
                held[i] = [x for x, m in zip(held[i], mask) if m]
                assert pool.seq_get(i)[0] == len(held[i])
                assert torch.equal(weights[i, :len(held[i])].cpu(), torch.from_numpy(w[mask == 1]))
                assert not weights[i, len(held[i]):].any()
    kvs = L.KvsMask(0)
    death, status = kvs.death_times([(lens[i], logs[i]) for i in range(n)], T)
    assert not status.any()
    # the engine rotates by position; the trainer takes the rotated queries and keys
    qr, kr = rotated[1].requires_grad_(), rotated[0].requires_grad_()
    vr = v.clone().requires_grad_()
    out = kvs.attention(qr, kr, vr, death, cap=cap)
    for i in range(n):
        a, b = out[i, :lens[i]].float(), served[i, :lens[i]].float()
        assert (a - b).abs().max() <= 4 * 2.0 ** -8 * float(v[i].float().abs().max())
    dout = randn(n, T, heads, dim)
    for i in range(n):
        dout[i, lens[i]:] = 0
    out.backward(dout)
    for i in range(n):
        seen = W.death_seen(death[i].cpu().numpy())
        f = lambda x: x.detach()[i].double().cpu().numpy()   # noqa: E731
        want = [np.zeros((T, heads, dim)), np.zeros((T, Hk, dim)), np.zeros((T, Hk, dim))]
        for h in range(heads):
            dq, dk, dv = W.gradients(f(qr)[:, h], f(kr)[:, h // G], f(vr)[:, h // G], f(dout)[:, h], seen, dim ** -0.5, cap)
            want[0][:, h] = dq
            want[1][:, h // G] += dk
            want[2][:, h // G] += dv
        for x, y in zip((qr, kr, vr), want):
            got = x.grad[i].double().cpu().numpy()
            assert np.linalg.norm(got - y) <= 4 * 2.0 ** -8 * np.linalg.norm(y)
            assert np.isfinite(got).all()
    kvs.close()
    step.close()
    pool.close()
