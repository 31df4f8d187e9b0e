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
