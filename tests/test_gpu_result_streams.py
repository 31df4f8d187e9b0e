"""Results that a call on another stream allocates: the current stream still has
work queued on a block of their size that has just been given back."""

import numpy as np
import pytest

from gpu_common import need_gpu, say, torch
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
