"""Death times at the ends of int32: a key that nobody sees is one whatever its death time
says, down to the bits of the gradients."""

import numpy as np
import pytest

from gpu_common import need_gpu, torch
from test_gpu_train import randn

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dead", [-2 ** 31, -2 ** 31 + 5, -1])
@pytest.mark.parametrize("T,H,G,D", [(4096, 1, 1, 64), (2500, 1, 2, 128)])
def test_the_least_death_times(T, H, G, D, dead):
    """Long tiles of keys are cut into shares by the work that the scan counts: keys that
    nobody sees are none of it."""
    L = need_gpu()
    kvs = L.KvsMask(0)
    g = np.random.default_rng(T)
    q, k, v, dout = randn(g, 1, T, H * G, D), randn(g, 1, T, H, D), randn(g, 1, T, H, D), randn(g, 1, T, H * G, D)
    results = []
    for value in (0, dead):
        death = torch.full((1, T), T, dtype=torch.int32, device="cuda")
        death[0, 7:2000:100] = value
        out, lse = kvs.attend(q, k, v, death)
        results.append((out, lse, *kvs.attend_backward(dout, q, k, v, out, lse, death)))
    for a, b in zip(*results):
        assert torch.equal(a, b)
    kvs.close()
