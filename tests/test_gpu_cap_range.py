"""Scales far above the cap, as the calls allow them, for queries whose scores are 0 or
far below it: the tanh's short form must not overflow.  Tolerances are those of
test_gpu_weight.py and test_gpu_train.py."""

import numpy as np
import pytest

from gpu_common import need_gpu, torch
from test_gpu_step import F32, _cache, _queries
from test_gpu_train import run
from test_gpu_weight import check_capped, weights_of

pytestmark = pytest.mark.gpu

RANGE = [(2.0 ** 32, 2.0 ** 20), (-2.0 ** 50, 2.0 ** 40), (2.0 ** 31, 2.0 ** 20), (2.0 ** 28, 2.0 ** 40),
         (2.0 ** -52, 2.0 ** -40)]


@pytest.mark.parametrize("scale,cap", RANGE)
@pytest.mark.parametrize("gqa", [False, True])
@pytest.mark.parametrize("count,times", [(1, 0.0), (20, 0.0), (20, 2.0 ** -20)])
def test_serving(gqa, scale, cap, count, times):
    need_gpu()
    c = _cache(gqa, 2, 64, 16, [150], seed=3)
    step = c.pool.step(4, max_tokens=20)
    step.begin([0], [count], grow=False)
    q = _queries(c, count, 4) * times
    out, lse = step.attend(0, q, scale=scale, lse=True, cap=cap)
    assert torch.isfinite(out).all() and torch.isfinite(lse).all()
    assert check_capped(c, out, lse, q, [0], [count], scale, cap) <= 1
    w = torch.zeros(1, 150, device="cuda")
    step.weigh(0, q, lse, w, scale=scale, cap=cap)
    # A score is a float32 and so is lse, each half a step off, 2^-24 of its size; where that
    # is more than 1 (scores of 2^33 here, 512 off) exp(s - lse) may be any number or infinity.
    if 2 * F32 * float(lse.abs().max()) > 1:
        return
    got = w[0].double().cpu().numpy()
    assert np.isfinite(got).all()
    (want, tol), = weights_of(c, q, lse, [0], [count], scale, cap, True, 0, 4)
    assert (np.abs(got - want) <= tol + F32 * want).all()
    if times == 0.0:   # every row that a token sees gets the same of it
        seen = 150 - count + 1 + np.arange(count)
        even = np.array([(4.0 / seen[seen > j]).sum() for j in range(150)])
        assert np.abs(got - even).max() <= 1e-5
    step.close()
    c.pool.close()


@pytest.mark.parametrize("scale,cap", RANGE)
@pytest.mark.parametrize("dk,dv", [(64, 64), (128, 128), (192, 128), (256, 256)])
def test_training(dk, dv, scale, cap):
    run(1, 140, 1, 2, dk, dv, "cut", cap, scale, seed=7, times=0.0)
