"""What the handle-less entry points share: argument checks, and the device and stream a call
runs on."""
from __future__ import annotations

import torch

from . import _lib

DTYPES = {torch.bfloat16: _lib.MOE_BF16, torch.float32: _lib.MOE_FP32}


def check_tensor(name: str, t, device, shape: tuple, dtype) -> None:
    """`t` must be a contiguous CUDA tensor on `device` of the given shape and dtype."""
    if not isinstance(t, torch.Tensor) or t.device != device:
        raise ValueError(f"{name} must be a CUDA tensor on {device}")
    if t.dtype != dtype or t.shape != shape or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {list(shape)} {dtype} tensor")


def rows_of(name: str, t) -> tuple:
    """(device, rows, width, dtype) of a [rows, width] bf16 or fp32 CUDA tensor."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.dim() != 2 or t.dtype not in DTYPES or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous [rows, width] torch.bfloat16 or torch.float32 tensor")
    return t.device, t.shape[0], t.shape[1], t.dtype


# the current stream's handle without a Stream object around it, where torch has the call
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda index: torch.cuda.current_stream(index).cuda_stream)


class on_stream:
    """The call's device made current and, when `stream` is given, its stream too, so that what
    the call allocates belongs to the stream that uses it.  `inputs` then also are recorded on
    the stream: the allocator will not hand out their memory while the call still reads it."""

    __slots__ = ("device", "stream", "inputs", "ctx")

    def __init__(self, device, stream=None, inputs=()):
        self.device, self.stream, self.inputs, self.ctx = device, stream, inputs, None

    def __enter__(self) -> int:
        if self.stream is None:
            if torch.cuda.current_device() != self.device.index:
                self.ctx = torch.cuda.device(self.device)
                self.ctx.__enter__()
            return _raw_stream(self.device.index)
        if self.stream.device != self.device:
            raise ValueError(f"stream is on {self.stream.device}, the tensors are on {self.device}")
        if self.stream != torch.cuda.current_stream(self.device):
            for t in self.inputs:
                if t is not None:
                    t.record_stream(self.stream)
        self.ctx = torch.cuda.stream(self.stream)
        self.ctx.__enter__()
        return self.stream.cuda_stream

    def __exit__(self, *exc):
        if self.ctx is not None:
            self.ctx.__exit__(*exc)
        return False
