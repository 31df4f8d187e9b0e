"""Results that a call allocates belong to the stream that the call runs on: a
block of another stream may still have work of that stream queued on it, or be
handed out again by it while the call still writes.  Checked without a GPU: the
allocations of calls with stream= are watched, and the call itself goes to a
library handle that refuses it."""

import contextlib

import pytest
import torch

from mla_paged_cache_amd import leyline as L
from test_step_binding import fake_step, z


class Handle:
    """What a caller passes as stream=."""
    cuda_stream = 0


@pytest.fixture
def watched(monkeypatch):
    """[(what was allocated, the stream it was allocated on or None)]"""
    seen, current = [], []

    @contextlib.contextmanager
    def on(stream):
        current.append(stream)
        try:
            yield
        finally:
            current.pop()

    def watch(name):
        plain = getattr(torch, name)

        def call(*a, **k):
            seen.append((name, current[-1].cuda_stream if current else None))
            return plain(*a, **k)
        monkeypatch.setattr(torch, name, call)
    for name in ("empty", "zeros", "full"):
        watch(name)
    monkeypatch.setattr(torch.cuda, "stream", on)
    monkeypatch.setattr(L, "_stream_handle", lambda stream, device: 0)   # no device to ask
    monkeypatch.setattr(torch.cuda, "ExternalStream",
                        lambda handle, device=None: type("S", (), {"cuda_stream": handle})())
    return seen


@pytest.mark.parametrize("gqa", [False, True])
@pytest.mark.parametrize("stream", [Handle(), None])
def test_a_steps_results(watched, gqa, stream):
    s = fake_step(gqa)
    q, full = z(3, 6, 64), z(3, 6, 64 if gqa else 576)
    watched.clear()
    where = None if stream is None else 0
    with pytest.raises(L.LeylineError):
        s.append(0, q=q, stream=stream)
    assert watched == [("empty", where)]
    with pytest.raises(L.LeylineError):
        s.attend(0, full, scale=0.1, lse=True, stream=stream)
    assert watched == [("empty", where)] * 3


def fake_kvs():
    """A mask context without a device and with a NULL handle."""
    k = object.__new__(L.KvsMask)
    k._h, k.device, k._tdev = None, 0, torch.device("cpu")
    return k


def no_device_check(monkeypatch):
    monkeypatch.setattr(L.KvsMask, "_check_death", lambda self, death: None)


@pytest.mark.parametrize("stream", [Handle(), None])
def test_a_masks_results(watched, monkeypatch, stream):
    """The block mask's counts and indices are also filled before the call."""
    no_device_check(monkeypatch)
    k, death = fake_kvs(), torch.zeros((2, 128), dtype=torch.int32)
    watched.clear()
    where = None if stream is None else 0
    with pytest.raises(L.LeylineError):
        k.dense_mask(death, stream=stream)
    assert watched == [("empty", where)]
    watched.clear()
    with pytest.raises(L.LeylineError):
        k.block_mask(death, 128, 128, stream=stream)
    assert watched == [("zeros", where)] * 2 + [("full", where)] * 2
    logs = type("Logs", (L._Logs,), {"__init__": lambda self: None})()
    logs.n, logs.logs, logs.keep = 2, None, torch.zeros(1, dtype=torch.uint8)
    watched.clear()
    with pytest.raises(L.LeylineError):
        k.death_times(logs, 128, stream=stream)
    assert watched == [("empty", where)] * 2


@pytest.mark.parametrize("gqa", [False, True])
@pytest.mark.parametrize("stream", [Handle(), None])
def test_gathered_rows(watched, gqa, stream):
    p = object.__new__(L.GqaPool if gqa else L.Pool)
    p._h, p._dev, p.device, p.num_layers, p.gqa, p.heads, p.head_dim = None, 0, torch.device("cpu"), 2, gqa, 3, 64
    angles = torch.zeros(5, dtype=torch.int64)
    watched.clear()
    with pytest.raises(L.LeylineError):
        p.rope_rows(0, 0, angles, out=True, stream=stream)
    assert watched == [("empty", None if stream is None else 0)]
