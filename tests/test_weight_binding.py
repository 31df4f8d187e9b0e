"""Host-side checks of eviction by attention weight and of the trainer's attention that
need no GPU: the binding covers include/leyline_weight.h and include/leyline_train.h, its
packed descriptors are the headers' structs, NULL handles are refused, tensors that do
not fit are refused before any pointer reaches the library, and the float64 oracle is
torch's attention, its gradients torch's and differences'."""

import ctypes
import os
import re
import shutil
import struct
import subprocess

import numpy as np
import pytest
import torch

from mla_paged_cache_amd import leyline as L
from oracle import weight_oracle as W
from test_step_binding import fake_step, z

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.mark.parametrize("header,exports", [("leyline_weight.h", L.WEIGHT_EXPORTS), ("leyline_train.h", L.TRAIN_EXPORTS)])
def test_binding_covers_the_header(header, exports):
    text = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", header)).read(), flags=re.S)
    names = re.findall(r"^(?:ll_status|void)\s+([a-z_]+)\s*\(", text, flags=re.M)
    assert sorted(names) == sorted(exports) and len(names) == 3
    for n in names:
        assert getattr(L._lib, n).argtypes is not None
    assert not set(exports) & set(L.EXPORTS + L.STEP_EXPORTS)


HEADS = ["{}.data", "{}.rollout_stride", "{}.token_stride", "{}.head_stride"]
TRAIN = ["n", "heads", "n_pad", "kv_heads", "key_dim", "value_dim", "scale", "cap", "death",
         *[h.format(x) for x in ("q", "k", "v", "out") for h in HEADS], "lse", "workspace", "workspace_bytes"]
FIELDS = {
    "ll_weigh_desc": (L._WEIGH_DESC.format, ["tokens", "layer", "causal", "window", "scale", "cap", "q", "q_token_stride",
                                             "q_head_stride", "q_pe", "q_pe_token_stride", "q_pe_head_stride", "lse",
                                             "weights", "weight_stride", "decay"]),
    "kvs_attend_desc": (L._TRAIN_DESC.format, TRAIN),
    "kvs_attend_backward_desc": (L._TRAIN_DESC.format + L._TRAIN_GRADS.format[1:],
                                 ["f." + f for f in TRAIN] + [h.format(x) for x in ("dout", "dq", "dk", "dv") for h in HEADS]),
}


def test_packed_descriptors_are_the_structs(tmp_path):
    """Each field's offset and the struct's size, from a compiler, against the places
    where the packed format puts 1, 2, 3, ..."""
    cc = shutil.which("gcc") or shutil.which("cc")
    if not cc:
        pytest.skip("no C compiler")
    lines = []
    for name, (_, fields) in FIELDS.items():
        lines.append(f'printf("{name} %zu\\n", sizeof({name}));')
        lines += [f'printf("%zu %zu\\n", offsetof({name}, {f}), sizeof((({name}*)0)->{f}));' for f in fields]
    src = tmp_path / "layout.c"
    src.write_text('#include <stddef.h>\n#include <stdio.h>\n#include "leyline_weight.h"\n#include "leyline_train.h"\n'
                   "int main(void) {\n" + "\n".join(lines) + "\nreturn 0;\n}\n")
    exe = tmp_path / "layout"
    subprocess.run([cc, f"-I{ROOT}/include", str(src), "-o", str(exe)], check=True)
    out = iter(subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout.splitlines())
    for name, (fmt, fields) in FIELDS.items():
        assert next(out) == f"{name} {struct.calcsize(fmt)}"
        data = struct.pack(fmt, *range(1, len(fields) + 1))
        for i, f in enumerate(fields):
            off, size = map(int, next(out).split())
            kind = "f" if f.split(".")[-1] in ("scale", "cap", "decay") else {4: "i", 8: "q"}[size]
            assert struct.unpack_from(kind, data, off)[0] == i + 1, f


def train_desc(n=1, heads=4, n_pad=100, kv_heads=2, dk=64, dv=64):
    d = L._TRAIN_DESC.pack(n, heads, n_pad, kv_heads, dk, dv, 1.0, 0.0, *[0] * 20)
    return d


def test_null_handles_are_refused():
    assert L._lib.ll_step_attend_capped(None, None, 1.0, None) == L.LL_EINVAL
    assert L._lib.ll_step_weigh(None, None, None) == L.LL_EINVAL
    assert L._lib.ll_keep_heaviest(None, None, 0, None, 0, 0, None, None, 0, None, None, None) == L.LL_EINVAL
    assert L._lib.kvs_attend(None, train_desc(), None) == L.LL_EINVAL
    assert L._lib.kvs_attend_backward(None, train_desc(), None) == L.LL_EINVAL
    assert "NULL" in L._lib.ll_last_error().decode()
    size = ctypes.c_int64()
    assert L._lib.kvs_attend_workspace(None, 0, ctypes.byref(size)) == L.LL_EINVAL
    assert L._lib.kvs_attend_workspace(train_desc(), 2, ctypes.byref(size)) == L.LL_EINVAL


def test_workspace_sizes():
    size = ctypes.c_int64()
    for back in (0, 1):
        last = 0
        for n_pad in (1, 64, 65, 4096, 100000):
            assert L._lib.kvs_attend_workspace(train_desc(n_pad=n_pad), back, ctypes.byref(size)) == L.LL_OK
            assert size.value >= last and size.value % 256 == 0
            last = size.value
    for bad in (dict(n=-1), dict(heads=0), dict(heads=3), dict(n_pad=0), dict(n_pad=2 ** 31 - 1), dict(kv_heads=0),
                dict(dk=0), dict(dk=12), dict(dv=264)):
        assert L._lib.kvs_attend_workspace(train_desc(**bad), 0, ctypes.byref(size)) == L.LL_EINVAL, bad


class FakePool:
    max_seqs, device = 2, torch.device("cpu")
    _weights = L.Pool._weights


@pytest.mark.parametrize("gqa", [False, True])
def test_weigh_checks_its_tensors(gqa):
    s = fake_step(gqa)
    s._pool = FakePool()
    q = z(3, 6, 64 if gqa else 576)
    lse, w = z(3, 6, dtype=torch.float32), z(2, 50, dtype=torch.float32)
    with pytest.raises(L.LeylineError):      # past the binding: the library refuses the NULL step
        s.weigh(0, q, lse, w, scale=0.1, cap=3.0, decay=0.5)
    with pytest.raises(L.LeylineError):
        s.attend(0, q, scale=0.1, cap=3.0)
    for kw in (dict(q=q.float()), dict(q=None), dict(lse=z(3, 6)), dict(lse=z(3, 5, dtype=torch.float32)),
               dict(lse=z(3, 12, dtype=torch.float32)[:, :6]), dict(lse=None), dict(weights=w[:1]), dict(weights=w.double()),
               dict(weights=z(2, 99, dtype=torch.float32)[:, :50]), dict(weights=w.to("meta")), dict(weights=None),
               dict(window=1.5), dict(scale="x"), dict(cap="x"), dict(decay="x"), dict(layer=1 << 31)):
        with pytest.raises(ValueError):
            s.weigh(**{"layer": 0, "q": q, "lse": lse, "weights": w, "scale": 0.1, **kw})


# ---- the oracle against torch and differences

@pytest.mark.parametrize("cap", [0.0, 1.3])
def test_oracle_attention_and_gradients(cap):
    g = np.random.default_rng(1)
    T, dk, dv = 11, 8, 6
    q, k, v, dout = (g.standard_normal((T, d)) for d in (dk, dk, dv, dv))
    death = np.array([1, 1, 4, 9, 4, 11, 7, 8, 11, 10, 11])   # query 1 sees nothing
    seen = W.death_seen(death)
    blind = ~seen.any(1)
    assert blind.any() and seen.any()
    a = [torch.from_numpy(x).requires_grad_() for x in (q, k, v)]

    def plain(q, k, v):
        x = 0.4 * q @ k.T
        x = cap * torch.tanh(x / cap) if cap else x
        x = x.masked_fill(torch.from_numpy(~seen), float("-inf"))[torch.from_numpy(~blind)]
        return torch.softmax(x, -1) @ v

    o = plain(*a)
    out, lse, weight, slack = W.attend(q, k, v, seen, 0.4, cap)
    np.testing.assert_allclose(out[~blind], o.detach().numpy(), rtol=1e-12, atol=1e-12)
    assert not out[blind].any() and np.isneginf(lse[blind]).all()
    (o * torch.from_numpy(dout[~blind])).sum().backward()
    for got, want in zip(W.gradients(q, k, v, dout, seen, 0.4, cap), a):
        np.testing.assert_allclose(got, want.grad.numpy(), rtol=1e-10, atol=1e-12)
    e, grads = 1e-6, W.gradients(q, k, v, dout, seen, 0.4, cap)
    for i in range(3):
        u = g.standard_normal(grads[i].shape)
        f = [float((W.attend(*[x + s * e * u if j == i else x for j, x in enumerate((q, k, v))], seen, 0.4, cap)[0] * dout).sum())
             for s in (1, -1)]
        assert abs((f[0] - f[1]) / (2 * e) - (grads[i] * u).sum()) < 1e-6
    w, _, _ = W.weigh(q, k, lse, seen, 0.4, cap)
    np.testing.assert_allclose(w.sum(), (~blind).sum(), rtol=1e-12)


def test_oracle_selection():
    w = np.array([1, 5, 5, np.nan, 0, -0.0, -3, np.inf, 5, 2], np.float32)
    assert list(np.flatnonzero(W.keep_heaviest(w, 3, 0, 0))) == [1, 3, 7]
    assert list(np.flatnonzero(W.keep_heaviest(w, 5, 1, 1))) == [0, 1, 3, 7, 9]
    assert list(np.flatnonzero(W.keep_heaviest(w, 8, 0, 0))) == [0, 1, 2, 3, 4, 7, 8, 9]
    assert W.keep_heaviest(w, 99, 2, 2).sum() == 10 and not W.keep_heaviest(w, 0, 0, 0).any()
