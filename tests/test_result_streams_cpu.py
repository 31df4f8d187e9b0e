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
