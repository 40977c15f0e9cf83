"""Tensors used on another stream than the one they were allocated on.

torch hands a freed tensor's memory out again on its own stream at once. A
call on a ``stream`` of its own may still be reading or writing it then, so
such a call marks every tensor it is given (and a workspace it makes) as used
on that stream. Calls on torch's current stream need none of this.
"""
import functools
import inspect

import torch


def _mark(v, stream):
    if isinstance(v, torch.Tensor):
        v.record_stream(stream)
    elif isinstance(v, (list, tuple)):
        for x in v:
            _mark(x, stream)


def lends(f):
    """Decorator of an entry point with a ``stream`` argument."""
    at = list(inspect.signature(f).parameters).index("stream")

    @functools.wraps(f)
    def call(*args, **kw):
        result = f(*args, **kw)
        stream = kw.get("stream") if len(args) <= at else args[at]
        if stream is not None:
            _mark(args, stream)
            _mark(list(kw.values()), stream)
        return result

    return call


def fresh(nbytes, device, stream):
    """A workspace of a call on ``stream`` (None: torch's current one)."""
    t = torch.empty(nbytes, dtype=torch.uint8, device=device)
    if stream is not None:
        t.record_stream(stream)
    return t
