"""Results that a call on another stream allocates: the current stream still has
work queued on a block of their size that has just been given back."""

import numpy as np
import pytest

from gpu_common import need_gpu, say, torch
from test_gpu_kvs_mask import _logs
from test_gpu_step import Cache, _queries, bf16, f64

pytestmark = pytest.mark.gpu


def queue_a_write(shapes):
    """Some milliseconds of work on the current stream, then writes of blocks of
    these shapes and types, which go back to the allocator at once."""
    need_gpu()
    x = torch.ones((4096, 4096), dtype=torch.bfloat16, device="cuda")
    y = torch.empty_like(x)
    for _ in range(40):
        torch.mm(x, x, out=y)
    blocks = [torch.full(s, 7, dtype=dt, device="cuda") for s, dt in shapes]
    del blocks


@pytest.mark.parametrize("gqa", [False, True])
def test_a_steps_results(gqa):
    say(f"results on another stream, gqa={gqa}")
    c = Cache(gqa, 16, [500, 31], seed=2, kv_heads=1, dim=64, rot=64)
    heads = 4
    step = c.pool.step(heads, max_tokens=8)
    side = torch.cuda.Stream()
    T = step.begin([0, 1], [1, 2], grow=False)
    q = _queries(c, T, heads)
    pe = q if gqa else q[..., 512:]
    want_q = f64(step.append(0, q=pe))
    torch.cuda.synchronize()
    queue_a_write([(pe.shape, torch.bfloat16), ((T, heads, 64 if gqa else 512), torch.bfloat16), ((T, heads), torch.float32)])
    got_q = step.append(0, q=pe, stream=side)
    out, lse = step.attend(0, q, scale=0.1, lse=True, stream=side)
    torch.cuda.synchronize()
    assert np.array_equal(f64(got_q), want_q)
    c.check_attend(out, lse, q, [0, 1], [1, 2], 0, 0.1)
    step.close()
    c.pool.close()


def test_a_masks_results():
    """The block mask's indices are filled before the call, on the same stream."""
    L = need_gpu()
    rolls = _logs(0, [256, 200, 131], ["window", "half", "pick"], budget=120, turn_lo=4, turn_hi=40, every=3)
    ctx, side = L.KvsMask(0), torch.cuda.Stream()
    death, status = ctx.death_times(rolls, 256)
    lists, bits = ctx.block_mask(death, 16, 16), ctx.dense_mask(death)
    torch.cuda.synchronize()
    i32 = torch.int32
    queue_a_write([(t.shape, i32) for t in (death, status, *lists, bits)])
    got = [*ctx.death_times(rolls, 256, stream=side), *ctx.block_mask(death, 16, 16, stream=side),
           ctx.dense_mask(death, stream=side)]
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(got, (death, status, *lists, bits)))
    ctx.close()


def test_gathered_rows():
    c = Cache(False, 16, [300], seed=2, layers=2)
    side = torch.cuda.Stream()
    angles = torch.arange(300, dtype=torch.int64, device="cuda")
    want = c.pool.rope_rows(0, 0, angles, out=True)
    torch.cuda.synchronize()
    queue_a_write([(want.shape, torch.bfloat16)])
    got = c.pool.rope_rows(0, 0, angles, out=True, stream=side)
    torch.cuda.synchronize()
    assert torch.equal(got.view(torch.int16), want.view(torch.int16))
    c.pool.close()
