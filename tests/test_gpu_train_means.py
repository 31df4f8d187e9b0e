"""Gradients of the trainer's attention where the queries' gradient is a small rest of
large terms: keys and values with a mean of their own (a projection with a bias), one key
that holds nearly all weight wherever it lies, and a query whose gradient is NaN beside
others that need the correction.

Tolerances, in 2-norm.  p or ds, and the result, are rounded to bf16: each is off by at
most half a step (2^-8 relative), evenly spread over it (2^-8 / sqrt(3) of the norm), the
two independently: 2^-8 sqrt(2/3).  What ds is rounded by counts for dq with its key's
distance from the query's weighted mean key, as ds itself does (its sum is 0), so a mean
of the keys adds nothing.  Everything else is float32."""

import numpy as np
import pytest

from gpu_common import need_gpu, torch
from test_gpu_operator_range import exact, off
from test_gpu_train import randn

pytestmark = pytest.mark.gpu

GRAD = 2.0 ** -8 * (2 / 3) ** 0.5


def documents(T, doc):
    t = np.arange(T)
    return torch.from_numpy(np.minimum((t // doc + 1) * doc, T).astype(np.int32)[None]).cuda()


def compare(L, q, k, v, dout, death, cap=0.0):
    kvs = L.KvsMask(0)
    out, lse = kvs.attend(q, k, v, death, cap=cap)
    got = kvs.attend_backward(dout, q, k, v, out, lse, death, cap=cap)
    errors = [off(a, b) for a, b in zip(got, exact(q, k, v, dout, death, q.shape[-1] ** -0.5, cap))]
    print(" ".join(f"{n} {e:.5f}" for n, e in zip(("dq", "dk", "dv"), errors)), flush=True)
    kvs.close()
    assert max(errors) <= GRAD, errors


@pytest.mark.parametrize("cap", [0.0, 30.0])
@pytest.mark.parametrize("T,H,G,dk,dv,doc,mean_k,mean_v", [
    (1024, 1, 2, 128, 128, 1024, 3.0, 0.0), (2048, 1, 1, 128, 128, 2048, 3.0, 0.6), (1500, 2, 1, 192, 128, 1500, 3.0, 0.3),
    (700, 2, 2, 64, 64, 700, 6.0, 0.6), (600, 1, 1, 256, 256, 600, 3.0, 1.0), (1200, 1, 3, 96, 96, 100, 3.0, 1.0),
    (389, 1, 2, 128, 64, 20, 5.0, 0.6), (131, 1, 1, 40, 72, 131, 3.0, 3.0)])
def test_keys_and_values_with_a_mean(T, H, G, dk, dv, doc, mean_k, mean_v, cap):
    """The same shift of every key: softmax and dq do not feel it without a cap."""
    L = need_gpu()
    g = np.random.default_rng(T)
    q, dout = randn(g, 1, T, H * G, dk), randn(g, 1, T, H * G, dv)
    k = (randn(g, 1, T, H, dk).float() + mean_k * randn(g, 1, 1, H, dk).float()).bfloat16()
    v = (randn(g, 1, T, H, dv).float() + mean_v * randn(g, 1, 1, H, dv).float()).bfloat16()
    compare(L, q, k, v, dout, documents(T, doc), cap)


@pytest.mark.parametrize("T,H,G,dk,dv,row,cap", [
    (2048, 1, 2, 128, 128, 10, 0.0), (2048, 1, 2, 128, 128, 70, 0.0), (1300, 1, 1, 192, 128, 100, 0.0),
    (1300, 1, 1, 192, 128, 70, 50.0), (1100, 2, 1, 64, 64, 65, 0.0), (1100, 1, 1, 256, 256, 127, 0.0),
    (4096, 1, 1, 128, 128, 70, 0.0)])
def test_one_key_with_nearly_all_weight(T, H, G, dk, dv, row, cap):
    """Of every query behind it; blocks of 64 keys count even or odd."""
    L = need_gpu()
    g = np.random.default_rng(T + row)
    q, k, v = randn(g, 1, T, H * G, dk), randn(g, 1, T, H, dk), randn(g, 1, T, H, dv)
    dout = randn(g, 1, T, H * G, dv)
    q[..., 0], k[..., 0] = 4.0, 0.0
    k[0, row, :, 0] = (np.log(T) + 6.0) / 4.0 * dk ** 0.5
    x = q[0, -200:, 0].double() @ k[0, :, 0].double().t().contiguous() * dk ** -0.5
    x = cap * torch.tanh(x / cap) if cap else x
    x.masked_fill_(torch.arange(T, device="cuda") > torch.arange(T - 200, T, device="cuda")[:, None], -1e300)
    p = torch.softmax(x, 1)[:, row]
    assert 0.9 < float(p.median()) < 0.9995
    compare(L, q, k, v, dout, documents(T, T), cap)


@pytest.mark.parametrize("T,dk,dv,doc,cap", [(390, 128, 128, 3, 0.0), (300, 64, 64, 2, 0.0), (300, 192, 128, 5, 30.0),
                                             (260, 256, 256, 4, 0.0)])
def test_a_gradient_of_nan_stays_with_its_query(T, dk, dv, doc, cap):
    """One query's dout, and another's out, hold NaN: the other queries' dq, and dk and dv
    of the keys that those two do not see, keep their bits."""
    L = need_gpu()
    g = np.random.default_rng(T)
    kvs = L.KvsMask(0)
    q, k, v, dout = randn(g, 1, T, 2, dk), randn(g, 1, T, 1, dk), randn(g, 1, T, 1, dv), randn(g, 1, T, 2, dv)
    death = documents(T, doc)
    out, lse = kvs.attend(q, k, v, death, cap=cap)
    want = kvs.attend_backward(dout, q, k, v, out, lse, death, cap=cap)
    dout, out = dout.clone(), out.clone()
    dout[0, 40, 0, 3] = float("nan")
    out[0, 171, 1, 5] = float("nan")
    got = kvs.attend_backward(dout, q, k, v, out, lse, death, cap=cap)
    rest = torch.ones(q.shape[:3], dtype=torch.bool, device="cuda")
    rest[0, 40, 0] = rest[0, 171, 1] = False
    assert torch.isnan(got[0][~rest]).all()
    assert torch.equal(got[0][rest], want[0][rest])
    t = torch.arange(T, device="cuda")
    unseen = (t // doc != 40 // doc) & (t // doc != 171 // doc)
    # (tiles that hold the NaN are done row by row, whose float32 sums have another order)
    for a, b in zip(got[1:], want[1:]):
        assert torch.isfinite(a[0, unseen]).all() and off(a[:, unseen], b[:, unseen].double()) <= 2 * GRAD
    kvs.close()
