"""Which stream a call runs on, and whose new tensors are."""
from __future__ import annotations

import contextlib

import torch

_HERE = contextlib.nullcontext()
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def enter(device: torch.device, stream):
    """The CUDA stream handle to enqueue on, and a context for the call: inside it ``device`` is the current device and
    new tensors belong to the stream (the given one, or the device's current one)."""
    if stream is None and device.index == torch.cuda.current_device():
        return (_raw_stream(device.index) if _raw_stream else torch.cuda.current_stream().cuda_stream), _HERE
    s = stream if stream is not None else torch.cuda.current_stream(device)
    if s.device != device:
        raise ValueError(f"the stream belongs to {s.device} and the tensors to {device}")
    ctx = contextlib.ExitStack()
    ctx.enter_context(torch.cuda.device(device))
    ctx.enter_context(torch.cuda.stream(s))
    return s.cuda_stream, ctx


def read_here(device: torch.device, *tensors: torch.Tensor | None) -> None:
    """Marks tensors of other streams as read by what the current stream (that of the call, inside its context) has enqueued:
    their memory is not handed out before that is done, even if they are dropped as soon as the call returns."""
    used = torch.cuda.current_stream(device)
    for t in tensors:
        if t is not None:
            t.record_stream(used)
