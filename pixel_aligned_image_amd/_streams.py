"""Tensors used on another stream than the one they were allocated on.

torch hands a freed tensor's memory out again on its own stream at once. A
call on a ``stream`` of its own may still be reading or writing it then, so
such a call marks every tensor it is given as used on that stream, and a
workspace that it makes is that stream's own. Calls on torch's current stream
need none of this.
"""
import functools
import inspect

import torch


def _as_torch(stream):
    """What torch knows as the stream of a call: the calls take any object
    with a ``cuda_stream`` handle."""
    if stream is None or isinstance(stream, torch.cuda.Stream):
        return stream
    return torch.cuda.ExternalStream(stream.cuda_stream)


def _mark(v, stream):
    if isinstance(v, torch.Tensor):
        if v.is_cuda:                        # (cameras may come as a CPU tensor)
            v.record_stream(stream)
    elif isinstance(v, (list, tuple)):
        for x in v:
            _mark(x, stream)


def lends(f):
    """Decorator of an entry point with a ``stream`` argument."""
    at = list(inspect.signature(f).parameters).index("stream")

    @functools.wraps(f)
    def call(*args, **kw):
        stream = _as_torch(kw.get("stream") if len(args) <= at else args[at])
        result = f(*args, **kw)
        if stream is not None:
            _mark(args, stream)
            _mark(list(kw.values()), stream)
        return result

    return call


def fresh(nbytes, device, stream):
    """A workspace of a call on ``stream`` (None: torch's current one). It is
    allocated on that stream: a block of the current stream may be one that
    was freed there while kernels which still use it are queued, and a call on
    another stream does not wait for them. Freed, it goes back to the stream
    that uses it."""
    if stream is None:
        return torch.empty(nbytes, dtype=torch.uint8, device=device)
    with torch.cuda.stream(_as_torch(stream)):
        return torch.empty(nbytes, dtype=torch.uint8, device=device)
