"""Which stream a call's tensors belong to, with the streams and the allocator
replaced by records of what was asked of them. CPU only."""
import contextlib

import pytest
import torch

from pixel_aligned_image_amd import _streams


class Recorder:
    """torch's current stream, and every allocation with the stream it was
    made on."""

    def __init__(self):
        self.current, self.made = "current", []

    @contextlib.contextmanager
    def stream(self, s):
        before, self.current = self.current, s
        yield
        self.current = before

    def empty(self, nbytes, dtype=None, device=None):
        self.made.append((nbytes, self.current))
        return self

    def record_stream(self, s):
        pass


@pytest.fixture
def recorder(monkeypatch):
    r = Recorder()
    monkeypatch.setattr(torch.cuda, "stream", r.stream)
    monkeypatch.setattr(torch, "empty", r.empty)
    return r


def test_fresh_workspaces_are_allocated_on_the_stream_that_uses_them(recorder):
    """A block of the current stream may still be in use there by kernels that
    a call on another stream does not wait for."""
    own = object()
    _streams.fresh(256, "cuda", own)
    _streams.fresh(512, "cuda", None)
    assert recorder.made == [(256, own), (512, "current")]
    assert recorder.current == "current"
