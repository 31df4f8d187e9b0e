"""Tensors of no tokens: their strides say nothing (torch gives those that come from
numpy strides of 0), so a step of no tokens takes them.  Without a device: calls
that pass the binding's checks reach the library, which refuses the NULL step."""

import numpy as np
import pytest
import torch

from mla_paged_cache_amd import leyline as L
from test_step_binding import fake_step, z


def empty(*tail, dtype=torch.bfloat16):
    t = torch.from_numpy(np.zeros((0, *tail), np.float32)).to(dtype)
    assert t.stride()[-1] == 0
    return t


@pytest.mark.parametrize("gqa", [False, True])
def test_no_tokens(gqa):
    s = fake_step(gqa)
    a, b = (empty(3, 64), empty(3, 64)) if gqa else (empty(512), empty(64))
    q, out = (empty(6, 64), empty(6, 64)) if gqa else (empty(6, 576), empty(6, 512))
    with pytest.raises(L.LeylineError):
        s.append(0, a, b, q=empty(6, 64), q_out=empty(6, 64))
    with pytest.raises(L.LeylineError):
        s.attend(0, q, scale=0.1, out=out, lse=empty(6, dtype=torch.float32))
    with pytest.raises(ValueError):   # other axes are refused all the same
        s.append(0, empty(3, 32), b)
    with pytest.raises(ValueError):
        s.attend(0, z(3, 6, 128 if gqa else 1152)[..., ::2], scale=0.1)
