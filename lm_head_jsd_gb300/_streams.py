"""The device and stream a call runs on, and its memory there."""
from __future__ import annotations

from contextlib import nullcontext

import torch

from . import _lib

_HERE = nullcontext()
_device = torch._C._cuda_getDevice if hasattr(torch._C, "_cuda_getDevice") else torch.cuda.current_device


def require_cuda(name, t):
    """Of a tensor or a device."""
    if not (t.is_cuda if isinstance(t, torch.Tensor) else t.type == "cuda"):
        raise ValueError(f"{name} is on {getattr(t, 'device', t)}, expected a CUDA device")


def on(stream, device):
    """Where a call allocates and launches: on ``stream`` (a Stream or its handle), so that
    what it takes is free there and what it drops is not handed out before that stream has
    passed the call; None: on the current stream of its tensors' device. A stream given by
    its handle must live as long as the results and the objects that were used on it."""
    if stream is None:
        return _HERE if device.index == _device() else torch.cuda.device(device)
    if not isinstance(stream, torch.cuda.Stream):
        handle = stream if isinstance(stream, int) else stream.cuda_stream
        # (0 and 1 are the default stream's)
        stream = (torch.cuda.default_stream(device) if handle in (0, 1)
                  else torch.cuda.ExternalStream(handle, device=device))
    return torch.cuda.stream(stream)


def hand_over(tensors, stream, device):
    """Results made on a given stream are the caller's: once dropped, their memory is not
    reused before the caller's current stream has passed its last use of them."""
    if stream is not None:
        caller = torch.cuda.current_stream(device)
        for t in tensors:
            if t is not None:
                t.record_stream(caller)


def capture_id():
    """Of the capture that the current stream is in; 0: none."""
    if not torch.cuda.is_current_stream_capturing():
        return 0
    return _lib.fljsd_capture_id()


def report(status, workspace, offset=0):
    """A call's status word into the caller's ``status``, on the current stream."""
    if status is not None:
        status.copy_(workspace[offset:offset + 4].view(torch.int32).view(status.shape))


def check_status(status, device):
    if status is not None and (status.dtype != torch.int32 or status.numel() != 1
                               or status.device != device):
        raise ValueError(f"status must be one int32 value on {device}")


class Memory:
    """Tensors that an object keeps from call to call, made on the stream that is current
    now: another stream's first use waits for what that one still does with their memory
    (its last user's work, or filling them), and it outlives the last use."""

    def __init__(self, tensors):
        self._tensors = tensors
        self._made = torch.cuda.current_stream(tensors[0].device)
        self._seen = {self._made.cuda_stream}

    def use(self):
        """Before a launch on the current stream."""
        if _lib._stream(None) in self._seen:
            return
        s = torch.cuda.current_stream(self._tensors[0].device)
        for t in self._tensors:
            t.record_stream(s)
        # (a capture may not wait for work outside of it, and starts when that has ended)
        if not torch.cuda.is_current_stream_capturing():
            s.wait_stream(self._made)
            self._seen.add(s.cuda_stream)
