"""The global 2-norm of many gradient tensors, and clipping to a given norm (moe_grad_* and
moe_clip_grad_norm in include/moe.h): N = sqrt(sum g^2), g *= min(1, max_norm / N).

When N is not finite the gradients stay as they are: the caller sees the norm.  The norm
stays on the device; nothing here waits for it.
"""
from __future__ import annotations

from array import array
from operator import attrgetter

import torch

from ._call import DTYPES, on_stream
from ._lib import check, lib


_device, _numel = torch.Tensor.get_device, torch.Tensor.numel
_address, _contiguous, _dtype = torch.Tensor.data_ptr, torch.Tensor.is_contiguous, attrgetter("dtype")


def _refuse(name: str, ts, dev) -> None:
    """Name the tensor the library cannot take."""
    for i, t in enumerate(ts):
        if not isinstance(t, torch.Tensor) or t.device != dev or t.dtype not in DTYPES or not t.is_contiguous():
            raise ValueError(f"{name}[{i}] must be a contiguous torch.bfloat16 or torch.float32 tensor on {dev}")


def _columns(name: str, ts, dev) -> tuple:
    """(addresses, element counts, library types) of the tensors; whole-list calls, since a
    model may have thousands of them."""
    try:
        good = set(map(_device, ts)) == {dev.index} and all(map(_contiguous, ts))
        types = list(map(DTYPES.get, map(_dtype, ts)))
    except TypeError:   # something that is no tensor
        good, types = False, [None]
    if not good or None in types:
        _refuse(name, ts, dev)
    # (lists first: an array grows with every element of an iterator)
    return array("Q", list(map(_address, ts))), array("q", list(map(_numel, ts))), array("i", types)


def _table(grads, outs=None):
    """(device, n, pointers, output pointers, element counts, dtypes) for the library; the
    arrays behind the pointers come last and have to outlive the call."""
    n = len(grads)
    if n == 0:
        raise ValueError("no gradients")
    dev = grads[0].device if isinstance(grads[0], torch.Tensor) else None
    if dev is None or dev.type != "cuda":
        raise ValueError("grads must be CUDA tensors")
    src, numels, types = _columns("grads", grads, dev)
    dst = src
    if outs is not None:
        if len(outs) != n:
            raise ValueError(f"{len(outs)} outputs for {n} gradients")
        dst, out_numels, out_types = _columns("out", outs, dev)
        if out_numels != numels or out_types != types:
            raise ValueError("each output must have as many elements as its gradient, and its type")
    return (dev, n, *(a.buffer_info()[0] for a in (src, dst, numels, types)), (src, dst, numels, types))


def _workspace(n: int, dev) -> torch.Tensor:
    return torch.empty(lib().moe_grad_workspace(n) // 8, dtype=torch.float64, device=dev)


def grad_norm(grads, stream: torch.cuda.Stream | None = None) -> torch.Tensor:
    """The 2-norm [1] fp32 of all `grads` (contiguous bf16 or fp32 CUDA tensors) together."""
    grads = list(grads)
    dev, n, src, _, numels, dts, _keep = _table(grads)
    with on_stream(dev, stream, grads) as s:
        norm = torch.empty(1, dtype=torch.float32, device=dev)
        ws = _workspace(n, dev)
        check(lib().moe_grad_sumsq(src, numels, dts, n, None, norm.data_ptr(), ws.data_ptr(),
                                   ws.numel() * 8, s))
    return norm


def grad_sumsq(grads, stream: torch.cuda.Stream | None = None) -> torch.Tensor:
    """The sum of squares [1] fp64 of all `grads`: what ranks that hold parts of one model's
    gradients add up before scale_grads (parallel.clip_grad_norm does both)."""
    grads = list(grads)
    dev, n, src, _, numels, dts, _keep = _table(grads)
    with on_stream(dev, stream, grads) as s:
        sumsq = torch.empty(1, dtype=torch.float64, device=dev)
        ws = _workspace(n, dev)
        check(lib().moe_grad_sumsq(src, numels, dts, n, sumsq.data_ptr(), None, ws.data_ptr(),
                                   ws.numel() * 8, s))
    return sumsq


def scale_grads(grads, sumsq: torch.Tensor, max_norm: float, out=None,
                stream: torch.cuda.Stream | None = None) -> torch.Tensor:
    """Scale `grads` (in place, or into `out`, tensors of as many elements and the same types) so that a
    gradient whose sum of squares is `sumsq` [1] fp64 has at most `max_norm`; returns its norm
    [1] fp32."""
    grads, outs = list(grads), list(out) if out is not None else None
    dev, n, src, dst, numels, dts, _keep = _table(grads, outs)
    if not isinstance(sumsq, torch.Tensor) or sumsq.device != dev or sumsq.dtype != torch.float64 \
            or sumsq.numel() != 1:
        raise ValueError(f"sumsq must be a [1] torch.float64 tensor on {dev}")
    with on_stream(dev, stream, [*grads, *(outs or ()), sumsq]) as s:
        norm = torch.empty(1, dtype=torch.float32, device=dev)
        check(lib().moe_grad_scale(src, dst, numels, dts, n, sumsq.data_ptr(), float(max_norm),
                                   norm.data_ptr(), s))
    return norm


def clip_grad_norm(grads, max_norm: float, out=None, stream: torch.cuda.Stream | None = None) -> torch.Tensor:
    """Scale `grads` so that their 2-norm together is at most `max_norm`: in place, or into
    `out` (a list of tensors of as many elements and the same types).  Returns the norm before, [1] fp32."""
    grads, outs = list(grads), list(out) if out is not None else None
    dev, n, src, dst, numels, dts, _keep = _table(grads, outs)
    with on_stream(dev, stream, [*grads, *(outs or ())]) as s:
        norm = torch.empty(1, dtype=torch.float32, device=dev)
        ws = _workspace(n, dev)
        check(lib().moe_clip_grad_norm(src, dst, numels, dts, n, float(max_norm), norm.data_ptr(),
                                       ws.data_ptr(), ws.numel() * 8, s))
    return norm
