"""The trainer's attention at the ends of what its calls take: more short rollouts than one
dispatch of the scan holds, and more work than the calls take."""

import ctypes

import numpy as np
import pytest

from gpu_common import need_gpu, torch
from test_gpu_train import randn

pytestmark = pytest.mark.gpu


def test_more_rollouts_than_one_dispatch_holds():
    """2^22 + 300 rollouts of a token: a workgroup of 1024 work-items for each one's lists, two
    for the gradients.  A token that sees itself gets its value and passes its gradient on;
    one that sees nothing gets and passes zeros."""
    L = need_gpu()
    kvs = L.KvsMask(0)
    n = (1 << 22) + 300
    gen = torch.Generator(device="cuda").manual_seed(1)
    q, k, v, dout = (torch.randn((n, 1, 1, 8), generator=gen, device="cuda").bfloat16() for _ in range(4))
    death = (torch.rand((n, 1), generator=gen, device="cuda") < 0.7).to(torch.int32)
    sees = (death > 0)[:, :, None]
    out, lse = kvs.attend(q, k, v, death, scale=0.5)
    assert torch.equal(out, v * sees[..., None])
    want = torch.where(sees, 0.5 * (q.double() * k.double()).sum(-1), -float("inf"))
    # (a float32 sum of 8 products, and a logarithm of 1)
    assert torch.equal(torch.isneginf(lse), ~sees) and float((lse - want)[sees].abs().max()) <= 16 * 2.0 ** -24 * 100
    dq, dk, dv = kvs.attend_backward(dout, q, k, v, out, lse, death, scale=0.5)
    # p is exp2 of lse against itself: 2^-22 (1 + |s|) off, and rounded to bf16 once more with
    # the result
    assert float((dv.double() - (dout * sees[..., None]).double()).abs().max()) <= 2.0 ** -7 * float(dout.abs().max())
    assert torch.equal(dv != 0, (dout != 0) & sees[..., None])
    for x in (dq, dk):   # one key takes all weight: what is left of dout . v - delta is float32's
        assert float(x.abs().max()) <= 2.0 ** -20 * 8 * float(dout.abs().max() * v.abs().max() * torch.max(q.abs().max(), k.abs().max()))
        assert not x[~sees[:, 0, 0]].any()
    kvs.close()


def test_more_work_than_the_calls_take():
    L = need_gpu()
    size = ctypes.c_int64()
    for n, heads, n_pad in ((1 << 23, 1, 1), (1 << 17, 64, 1), (2, 1, 64 << 22), (1, 1 << 23, 5)):
        d = L._TRAIN_DESC.pack(n, heads, n_pad, 1, 8, 8, 1.0, 0.0, *[0] * 20)
        assert L._lib.kvs_attend_workspace(d, 1, ctypes.byref(size)) == L.LL_EUNSUPPORTED
    kvs = L.KvsMask(0)
    z = randn(np.random.default_rng(0), 1, 1, 1, 8)
    d = torch.ones((1, 1), dtype=torch.int32, device="cuda").expand(1 << 23, 1)
    with pytest.raises((L.LeylineError, ValueError)):
        kvs.attend(*[z.expand(1 << 23, 1, 1, 8)] * 3, d.contiguous(), out=z.expand(1 << 23, 1, 1, 8))
    kvs.close()
