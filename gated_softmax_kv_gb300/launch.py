"""What the bindings of rope.py and cache.py share around a launch: the
device, the stream, the life of the tensors and the overlap of an output."""
from __future__ import annotations

from .binding import _stream_handle


class on_device:
    """Makes `dev` the current device for a call and `stream` (None: the
    device's current stream) the one that outputs are allocated on. The common
    case, everything current already, switches nothing."""

    def __init__(self, dev: int, stream=None):
        import torch
        self._stream = stream
        self._guards = []
        if torch.cuda.current_device() != dev:
            self._guards.append(torch.cuda.device(dev))
        if stream is not None:
            self._guards.append(torch.cuda.stream(stream))
        self._dev = dev
        self.handle = 0

    def __enter__(self):
        for g in self._guards:
            g.__enter__()
        self.handle = _stream_handle(self._stream, self._dev)
        return self

    def __exit__(self, *exc):
        for g in reversed(self._guards):
            g.__exit__(*exc)
        return False

    def used(self, *tensors):
        """With a stream of the caller's choosing: the caching allocator must
        not hand a tensor's memory on before that stream is done with it."""
        if self._stream is not None:
            for t in tensors:
                if t is not None:
                    t.record_stream(self._stream)


def _span(t):
    """[first, last) byte addresses that the tensor's elements lie in."""
    if t.numel() == 0:
        return 0, 0
    first = t.data_ptr()
    last = first + t.element_size() * (1 + sum((n - 1) * s for n, s in zip(t.shape, t.stride())))
    return first, last


def output_overlaps(out, x) -> bool:
    """Whether out and x share memory without being the same elements."""
    if out.data_ptr() == x.data_ptr() and out.stride() == x.stride():
        return False
    a, b = _span(out)
    c, d = _span(x)
    return a < d and c < b
