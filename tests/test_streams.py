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


class Handle:
    """A stream of another library: a handle and nothing else."""
    cuda_stream = 0x1230


class Held(torch.Tensor):
    """A CPU tensor that says it is on the GPU and keeps its marks."""
    is_cuda = property(lambda self: True)

    def record_stream(self, s):
        self.marks.append(s)


@pytest.fixture
def external(monkeypatch):
    class External:
        def __init__(self, handle):
            self.cuda_stream = handle
    monkeypatch.setattr(torch.cuda, "ExternalStream", External)
    return External


def test_fresh_workspaces_are_allocated_on_the_stream_that_uses_them(recorder, external):
    """A block of the current stream may still be in use there by kernels that
    a call on another stream does not wait for."""
    _streams.fresh(256, "cuda", Handle)
    _streams.fresh(512, "cuda", None)
    assert [n for n, _ in recorder.made] == [256, 512]
    assert recorder.made[0][1].cuda_stream == Handle.cuda_stream
    assert recorder.made[1][1] == "current"
    assert recorder.current == "current"


def call(x, cams, weights=(), stream=None):
    return stream


def held():
    t = torch.zeros(2).as_subclass(Held)
    t.marks = []
    return t


@pytest.mark.parametrize("positional", [False, True])
def test_any_object_with_a_handle_is_a_stream(external, positional):
    """The calls read no more of a stream than its handle; so do the marks."""
    x, w = held(), held()
    lent = _streams.lends(call)
    got = lent(x, [], [w], Handle) if positional else lent(x, [], [w], stream=Handle)
    assert got is Handle                     # the call itself gets what was given
    for t in (x, w):
        assert [type(s) for s in t.marks] == [external]
        assert t.marks[0].cuda_stream == Handle.cuda_stream


def test_what_is_no_stream_is_refused_before_the_call(external):
    ran = []

    def enqueue(x, stream=None):
        ran.append(x)

    with pytest.raises(AttributeError):
        _streams.lends(enqueue)(held(), stream=7)
    assert not ran


def test_cpu_tensors_are_not_marked(external):
    """Cameras are any sequence of pairs, a CPU tensor's rows too."""
    _streams.lends(call)(held(), torch.zeros(1, 2), stream=Handle)
