"""What the bindings of rope.py and cache.py share around a launch: the
device, the stream, the life of the tensors, and an output of the caller's: its
overlap, and what autograd is told of it."""
from __future__ import annotations

from . import binding


class _Launch:
    """A launch on the device's current stream, which is where everything lives already."""

    __slots__ = ("handle",)

    def __init__(self, handle: int):
        self.handle = handle

    def __enter__(self):
        return self

    def __exit__(self, *exc):
        return False

    def used(self, *tensors):
        pass


class _GuardedLaunch(_Launch):
    """A launch on another device than the current one, or on a stream of the
    caller's choosing: both are current for the call, so that outputs are
    allocated there, and the caching allocator is told which tensors the
    stream uses before it may hand their memory on."""

    __slots__ = ("_stream", "_guards", "_dev")

    def __init__(self, dev: int, stream):
        import torch
        self._stream, self._dev = stream, dev
        self._guards = [torch.cuda.device(dev)]
        if stream is not None:
            self._guards.append(torch.cuda.stream(stream))

    def __enter__(self):
        for g in self._guards:
            g.__enter__()
        self.handle = binding._stream_handle(self._stream, self._dev)
        return self

    def __exit__(self, *exc):
        for g in reversed(self._guards):
            g.__exit__(*exc)
        return False

    def used(self, *tensors):
        if self._stream is not None:
            for t in tensors:
                if t is not None:
                    t.record_stream(self._stream)


_current_device = None


def on_device(dev: int, stream=None) -> _Launch:
    """The launch of a call on device `dev` and `stream` (None: the device's
    current stream), to be used as a context."""
    global _current_device
    if _current_device is None:
        import torch
        _current_device = torch.cuda.current_device
    if stream is None and _current_device() == dev:
        return _Launch(binding._stream_handle(None, dev))
    return _GuardedLaunch(dev, stream)


def changed(*tensors):
    """Tells autograd that a kernel wrote over tensors of the caller, so that a
    graph that saved their old values refuses its backward pass."""
    import torch
    torch.autograd.graph.increment_version(tensors)


def _span(t):
    """[first, last) byte addresses that the tensor's elements lie in."""
    if t.numel() == 0:
        return 0, 0
    first = t.data_ptr()
    last = first + t.element_size() * (1 + sum((n - 1) * s for n, s in zip(t.shape, t.stride())))
    return first, last


def output_overlaps(out, x) -> bool:
    """Whether out and x share memory without being the same elements."""
    if out is x or out.data_ptr() == x.data_ptr() and out.stride() == x.stride():
        return False
    a, b = _span(out)
    c, d = _span(x)
    return a < d and c < b
