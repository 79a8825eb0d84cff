"""What the classes that own device buffers share: work on the stream of a
call, and the memory that such work still reads or writes."""
from __future__ import annotations

import torch

from . import _stream


class StreamUser:
    """A class with a ``device`` whose calls take ``stream``: None (the current
    one), a torch stream or a raw handle."""

    _streams = _made = None

    def _ready(self):
        """The object is made: its buffers are filled, or may be memory that
        others used, by work of the current stream, which calls on other
        streams come after (_enter)."""
        self._streams, self._made = set(), None
        if self.device.type == "cuda":
            with torch.cuda.device(self.device):
                s = torch.cuda.current_stream()
                self._streams.add(s.cuda_stream)
                if not torch.cuda.is_current_stream_capturing():
                    self._made = s.record_event()

    def _enter(self, stream):
        """A call on `stream` begins, with the device current.  The first one on
        a stream comes after what made the object, and from then on the memory
        of its buffers is not given to others before that stream is done with
        it, though the object goes.  Not in a capture, which waits for nothing
        outside it and whose owner keeps what it uses."""
        if self._streams is None or self.device.type != "cuda":
            return
        handle = _stream(stream)
        if handle in self._streams:
            return
        s = torch.cuda.current_stream() if stream is None else self._torch_stream(stream)
        with torch.cuda.stream(s):
            if torch.cuda.is_current_stream_capturing():
                return
        self._streams.add(handle)
        if self._made is not None:
            s.wait_event(self._made)
        for t in self._buffers():
            t.record_stream(s)

    def _buffers(self):
        """The tensors that the object holds on its device."""
        found, more, where = [], list(vars(self).values()), self._where()
        while more:
            t = more.pop()
            if isinstance(t, (list, tuple)):
                more.extend(t)
            elif isinstance(t, torch.Tensor) and t.device == where:
                found.append(t)
        return found

    def _torch_stream(self, stream):
        """The torch stream of a call's `stream` (None: the current one, or a raw handle)."""
        if isinstance(stream, int):
            return torch.cuda.ExternalStream(stream, device=self.device)
        return stream

    def _after_current(self, stream, *new):
        """Work on `stream` waits for the current one: the buffers `new` may be
        memory that the current stream still works on."""
        s = self._torch_stream(stream)
        if s is not None and s != torch.cuda.current_stream():
            s.wait_stream(torch.cuda.current_stream())
        self._hold(stream, *new)

    def _hold(self, stream, *tensors):
        """Memory of tensors that work on `stream` reads or writes is not given
        to others before it is done, though every owner lets it go."""
        s = self._torch_stream(stream)
        if s is not None:
            for t in tensors:
                if t is not None:
                    t.record_stream(s)

    def _expect(self, what, t, dtype, shape):
        """Refuses a tensor that a kernel could not read as `shape` values of `dtype`."""
        if t.dtype != dtype or tuple(t.shape) != tuple(shape) or not t.is_contiguous() or t.device != self._where():
            raise ValueError(f"{what}: contiguous {dtype} {tuple(shape)} on {self._where()} expected, got {t.dtype} "
                             f"{tuple(t.shape)}{'' if t.is_contiguous() else ' (strided)'} on {t.device}")

    def _where(self):
        """The device with its number, as a tensor names it."""
        if self.device.type == "cuda" and self.device.index is None:
            return torch.device("cuda", torch.cuda.current_device())
        return self.device
