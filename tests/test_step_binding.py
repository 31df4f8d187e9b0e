"""Host-side checks of the serving step that need no GPU: the binding covers
include/leyline_step.h, its packed descriptors are the header's structs, NULL
handles are refused, and tensors of the wrong shape, type, layout or device are
refused with ValueError before any pointer reaches the library.  The float64
oracle is checked against torch on the side."""

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
from oracle import step_oracle as S

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "leyline_step.h")


def test_binding_covers_the_header():
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    names = re.findall(r"^(?:ll_status|void)\s+([a-z_]+)\s*\(", text, flags=re.M)
    assert sorted(names) == sorted(L.STEP_EXPORTS) and len(names) == 5
    for n in names:
        assert getattr(L._lib, n).argtypes is not None
    assert not set(L.STEP_EXPORTS) & set(L.EXPORTS)


FIELDS = {
    "ll_append_desc": (L._APPEND_DESC, ["tokens", "layer", "norm_type", "a", "a_token_stride", "a_head_stride", "b",
                                        "b_token_stride", "b_head_stride", "norm", "q", "q_token_stride", "q_head_stride",
                                        "q_out", "q_out_token_stride", "q_out_head_stride", "q_norm", "eps"]),
    "ll_attend_desc": (L._ATTEND_DESC, ["tokens", "layer", "causal", "window", "scale", "q", "q_token_stride",
                                        "q_head_stride", "q_pe", "q_pe_token_stride", "q_pe_head_stride", "out",
                                        "out_token_stride", "out_head_stride", "lse"]),
}


def test_packed_descriptors_are_the_structs(tmp_path):
    """Each field's offset and the struct's size, from a compiler, against the
    places where the packed format puts 1, 2, 3, ..."""
    cc = shutil.which("gcc") or shutil.which("cc")
    if not cc:
        pytest.skip("no C compiler")
    lines = []
    for name, (_, fields) in FIELDS.items():
        lines.append(f'printf("{name} %zu\\n", sizeof({name}));')
        lines += [f'printf("%zu %zu\\n", offsetof({name}, {f}), sizeof((({name}*)0)->{f}));' for f in fields]
    src = tmp_path / "layout.c"
    src.write_text('#include <stddef.h>\n#include <stdio.h>\n#include "leyline_step.h"\nint main(void) {\n'
                   + "\n".join(lines) + "\nreturn 0;\n}\n")
    exe = tmp_path / "layout"
    subprocess.run([cc, f"-I{ROOT}/include", str(src), "-o", str(exe)], check=True)
    out = iter(subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout.splitlines())
    for name, (fmt, fields) in FIELDS.items():
        assert next(out) == f"{name} {fmt.size}"
        data = fmt.pack(*range(1, len(fields) + 1))
        for i, f in enumerate(fields):
            off, size = map(int, next(out).split())
            kind = "f" if f in ("scale", "eps") else {4: "i", 8: "q"}[size]
            assert struct.unpack_from(kind, data, off)[0] == i + 1, f
    assert ctypes.sizeof(L._StepDesc) == 12


def test_null_handles_are_refused():
    d, h = L._StepDesc(8, 1, 1), ctypes.c_void_p(1)
    assert L._lib.ll_step_create(None, ctypes.byref(d), ctypes.byref(h)) == L.LL_EINVAL and not h.value
    assert L._lib.ll_step_begin(None, None, None, 0, 1, None) == L.LL_EINVAL
    assert L._lib.ll_step_append(None, None, None) == L.LL_EINVAL
    assert L._lib.ll_step_attend(None, None, None) == L.LL_EINVAL
    assert "NULL" in L._lib.ll_last_error().decode()
    L._lib.ll_step_destroy(None)


def fake_step(gqa, heads=6):
    """A step without a device: calls that pass the binding's checks reach the
    library, which refuses the NULL step."""
    s = object.__new__(L.Step)
    s._h, s._dev, s.device = None, 0, torch.device("cpu")
    s.gqa, s.heads, s.max_seqs, s.max_tokens, s.tokens = gqa, heads, 4, 64, 3
    s._dv, s._dr = (64, 64) if gqa else (512, 64)
    s._a_tail = (3, 64) if gqa else (512,)
    s._b_tail = (3, 64) if gqa else (64,)
    s._q_tail, s._r_tail, s._o_tail, s._l_tail = (heads, 576), (heads, s._dr), (heads, s._dv), (heads,)
    s._torch, s._bf16, s._f32, s._raw_stream = torch, torch.bfloat16, torch.float32, lambda d: 0
    return s


def z(*shape, dtype=torch.bfloat16):
    return torch.zeros(shape, dtype=dtype)


@pytest.mark.parametrize("gqa", [False, True])
def test_append_checks_its_tensors(gqa):
    s = fake_step(gqa)
    a, b = (z(3, 3, 64), z(3, 3, 64)) if gqa else (z(3, 512), z(3, 64))
    q, w = z(3, 6, 64), z(64 if gqa else 512)
    with pytest.raises(L.LeylineError):
        s.append(0, a, b, norm=w, q=q)
    with pytest.raises(L.LeylineError):
        s.append(0, a, b, norm=w.float(), q=q, q_out=q)
    bad = [dict(a=a), dict(b=b), dict(a=a, b=b.float()), dict(a=a[..., ::2], b=b), dict(a=b[:, :1], b=b),
           dict(a=a, b=np.zeros(b.shape)), dict(a=a, b=b, q=z(3, 5, 64)), dict(a=a, b=b, q=z(3, 6, 128)[..., ::2]),
           dict(a=a, b=b, q=q, q_out=z(3, 6, 32)), dict(a=a, b=b, q_out=q), dict(a=a, b=b, norm=z(8)),
           dict(a=a, b=b, norm=w.half()), dict(a=a, b=b, norm=z(2 * w.shape[0])[::2]),
           dict(a=a, b=b, q=q, q_out=3.0), dict(a=a, b=b, q=q.to("meta")), dict(a=a, b=b, q_norm=z(64)),
           dict(a=a, b=b, q=q, norm=w, q_norm=z(64).float()), dict(a=a, b=b, norm=1.0), dict(a=a, b=b, eps="x")]
    for kw in bad:
        with pytest.raises(ValueError):
            s.append(0, **kw)
    for layer in (1 << 31, 0.5, None):
        with pytest.raises(ValueError):
            s.append(layer, a, b)


@pytest.mark.parametrize("gqa", [False, True])
def test_attend_checks_its_tensors(gqa):
    s = fake_step(gqa)
    q, out = (z(3, 6, 64), z(3, 6, 64)) if gqa else (z(3, 6, 576), z(3, 6, 512))
    with pytest.raises(L.LeylineError):
        s.attend(0, q, scale=0.1, out=out, lse=True)
    bad = [dict(q=q.float()), dict(q=q[:, :5]), dict(q=q[..., :32]), dict(q=q.to("meta")), dict(q=None),
           dict(q=q, out=out.float()), dict(q=q, out=out[..., ::2]), dict(q=q, out=z(3, 6, 8)),
           dict(q=q, lse=z(3, 6)), dict(q=q, lse=z(3, 5, dtype=torch.float32)),
           dict(q=q, lse=z(3, 12, dtype=torch.float32)[:, :6])]
    bad += [dict(q=q, q_pe=z(3, 6, 64))] if gqa else [dict(q=z(3, 6, 512)), dict(q=z(3, 6, 512), q_pe=z(3, 6, 32)),
                                                       dict(q=q, q_pe=z(3, 6, 64))]
    for kw in bad:
        with pytest.raises(ValueError):
            s.attend(0, scale=0.1, **kw)
    for kw in (dict(window=1 << 63), dict(window=1.5), dict(scale="x"), dict(layer=1 << 31)):
        with pytest.raises(ValueError):
            s.attend(**{"layer": 0, "q": q, "scale": 0.1, **kw})
    if gqa:
        with pytest.raises(L.LeylineError):
            s.attend(0, q)            # the scale has a default
    else:
        with pytest.raises(ValueError):
            s.attend(0, q)
        with pytest.raises(L.LeylineError):
            s.attend(0, z(3, 6, 512), z(3, 6, 64), scale=0.1)


def test_begin_checks_its_lists():
    s = fake_step(False)
    with pytest.raises(ValueError):
        s.begin([0, 1], [1], stream=type("S", (), {"cuda_stream": 0})())
    with pytest.raises(L.LeylineError):
        s.begin([0, 1], [1, 1], stream=type("S", (), {"cuda_stream": 0})())


# ---- the oracle against torch

@pytest.mark.parametrize("causal,window", [(True, 0), (True, 3), (False, 0)])
def test_oracle_attention_is_softmax_attention(causal, window):
    g = np.random.default_rng(1)
    q, k, v = g.standard_normal((5, 8)), g.standard_normal((9, 8)), g.standard_normal((9, 6))
    out, lse, _, _ = S.attend(q, k, v, 4, 0.3, causal, window)
    i, j = np.arange(5)[:, None] + 4, np.arange(9)[None]
    seen = (j <= i) if causal else np.ones((5, 9), bool)
    if window:
        seen &= j > i - window
    x = torch.from_numpy(0.3 * q @ k.T).masked_fill(torch.from_numpy(~seen), float("-inf"))
    np.testing.assert_allclose(out, (torch.softmax(x, -1) @ torch.from_numpy(v)).numpy(), rtol=1e-12, atol=1e-12)
    np.testing.assert_allclose(lse, torch.logsumexp(x, -1).numpy(), rtol=1e-12)


@pytest.mark.parametrize("pairing", [0, 1])
def test_oracle_rotation_is_the_rotation_matrix(pairing):
    g = np.random.default_rng(2)
    x, ang = g.standard_normal((4, 2, 24)), S.angles([0, 1, 7, 123456], 16, 10000.0)
    got, size = S.heads(x, None, 0, ang, pairing, 16)
    for j in range(8):
        a, b = (2 * j, 2 * j + 1) if pairing == 0 else (j, j + 8)
        c, s = np.cos(ang[:, j])[:, None], np.sin(ang[:, j])[:, None]
        np.testing.assert_allclose(got[..., a], x[..., a] * c - x[..., b] * s, atol=1e-12)
        np.testing.assert_allclose(got[..., b], x[..., a] * s + x[..., b] * c, atol=1e-12)
    assert np.array_equal(got[..., 16:], x[..., 16:]) and (np.abs(got) <= size + 1e-12).all()
