"""What the operator classes share: a status word and a workspace on one
device, the stream that a call goes to, and their native calls."""
from __future__ import annotations

import importlib.machinery
import importlib.util
import os

import torch

from . import library_path
from ._build import CALLS

_raw_stream = torch._C._cuda_getCurrentRawStream
_current_device = torch._C._cuda_getDevice


def _load_calls():
    if not os.path.exists(CALLS):
        raise ImportError(f"{CALLS} is missing: build it with __graft_entry__.build() (it stands "
                          f"beside {library_path()}; there is no fallback)")
    loader = importlib.machinery.ExtensionFileLoader("_calls", CALLS)
    module = importlib.util.module_from_spec(importlib.util.spec_from_loader("_calls", loader))
    loader.exec_module(module)
    return module


calls = _load_calls()
NEEDS_WORKSPACE = -1         # of calls.packed: larger than the workspace was sized for


class DeviceOperator:
    """``dev_status`` collects the device's error bits (``SA_DEV_*``).  The
    calls of one object share its workspace: they must not run at the same time
    on several streams, nor may the replays of graphs that hold them.  A graph
    that captured a call needs the object, and its tensors, to live."""

    def __init__(self, device):
        dev = torch.device(device)
        if dev.type != "cuda":
            raise ValueError("the device must be a CUDA device")
        self._index = torch.cuda.current_device() if dev.index is None else dev.index
        self.device = torch.device("cuda", self._index)
        self.dev_status = torch.zeros(1, dtype=torch.int32, device=self.device)
        self._status = self.dev_status.data_ptr()
        self._ws, self._ws_ptr, self._ws_bytes = None, None, 0
        self._outgrown = []
        # the streams that the status word and the workspace were allocated on
        self._status_stream = self._ws_stream = _raw_stream(self._index)

    def _made(self):
        """The end of a constructor: what it queued, and what its memory's last
        owners had queued before, is done, so that a call may go to any stream."""
        with torch.cuda.device(self.device):
            if not torch.cuda.is_current_stream_capturing():
                torch.cuda.current_stream().synchronize()

    def _need(self, need):
        """A workspace of at least ``need`` bytes; the device is current."""
        if need <= self._ws_bytes:
            return
        if self._ws is not None:            # graphs captured with it still use it
            self._outgrown.append(self._ws)
        self._ws = torch.empty(need, dtype=torch.uint8, device=self.device)
        self._ws_ptr, self._ws_bytes = self._ws.data_ptr(), need
        self._ws_stream = _raw_stream(self._index)

    def _stream(self, stream):
        """The torch stream of a ``stream`` argument: a handle, or a stream of
        this device."""
        if isinstance(stream, int):
            # (an external stream of handle 0 would be a new stream)
            return (torch.cuda.ExternalStream(stream, device=self.device) if stream else
                    torch.cuda.default_stream(self.device))
        if stream.device_index != self._index:
            raise ValueError(f"stream must be on {self.device}")
        return stream

    def _handle(self):
        """The current stream's handle; the object's own tensors outlive the
        work of streams that they were not allocated on."""
        handle = _raw_stream(self._index)
        if handle != self._status_stream:
            self.dev_status.record_stream(self._stream(handle))
        if handle != self._ws_stream and self._ws is not None:
            self._ws.record_stream(self._stream(handle))
        return handle

    def _elsewhere(self, stream):
        """Whether a call has to go through ``_on``."""
        return stream is not None or _current_device() != self._index

    def _on(self, stream, call):
        """``call()`` with the device and ``stream`` (None: the current one)
        current; a tensor that it returns may be used on the caller's stream."""
        with torch.cuda.device(self.device):
            if stream is None:
                return call()
            caller, stream = torch.cuda.current_stream(), self._stream(stream)
            if stream.cuda_stream == caller.cuda_stream:
                return call()
            with torch.cuda.stream(stream):
                out = call()
            for t in out if isinstance(out, tuple) else (out,):
                if t is not None:
                    t.record_stream(caller)
            return out

    def _own(self, t, dtype, shape, name):
        """Address of a contiguous tensor of this device (None: NULL)."""
        if t is None:
            return None
        if t.dtype is not dtype or tuple(t.shape) != tuple(shape) or not t.is_contiguous():
            raise ValueError(f"{name} must be a contiguous {dtype} tensor of shape {list(shape)}")
        if t.get_device() != self._index:
            raise ValueError(f"{name} must be on {self.device}")
        return t.data_ptr()
