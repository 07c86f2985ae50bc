"""Matrix products grouped by expert over ragged rows (moe_grouped_* in include/moe.h).

Expert e owns counts[e] consecutive rows, experts in order and unpadded: the form in which
`LibEPBackend.dispatch` returns its rows and counts.  The three products are a linear layer
per expert, its input gradient and its weight gradient:

  grouped_mm        y[r] = x[r] W_e^T
  grouped_mm_dgrad  dx[r] = dy[r] W_e
  grouped_mm_wgrad  dW_e = dy_e^T x_e  (fp32, optionally added to what is there)

Argument marshalling only; the products run in libmoe.so.
"""
from __future__ import annotations

import torch

from ._call import DTYPES, check_tensor, on_stream, rows_of
from ._lib import check, lib


def _weights(w, device, dtype) -> tuple:
    if not isinstance(w, torch.Tensor) or w.dim() != 3:
        raise ValueError("w must be a [groups, n, k] tensor")
    check_tensor("w", w, device, tuple(w.shape), dtype)
    return tuple(w.shape)


def grouped_mm(x: torch.Tensor, w: torch.Tensor, counts: torch.Tensor, out: torch.Tensor | None = None,
               stream: torch.cuda.Stream | None = None) -> torch.Tensor:
    """y [rows, n]: each expert's rows of x [rows, k] times W_e^T, w [groups, n, k], counts
    [groups] int32 on the device.  Rows behind the last expert's are not written: they keep
    what `out` holds, and are unspecified without `out`."""
    dev, rows, k, dt = rows_of("x", x)
    g, n, wk = _weights(w, dev, dt)
    if wk != k:
        raise ValueError(f"x is {k} wide, w takes {wk}")
    check_tensor("counts", counts, dev, (g,), torch.int32)
    if out is not None:
        check_tensor("out", out, dev, (rows, n), dt)
    with on_stream(dev, stream, (x, w, counts, out)) as s:
        if out is None:
            out = torch.empty(rows, n, dtype=dt, device=dev)
        check(lib().moe_grouped_mm(x.data_ptr(), w.data_ptr(), counts.data_ptr(), g, rows, n, k,
                                   DTYPES[dt], out.data_ptr(), s))
    return out


def grouped_mm_dgrad(dy: torch.Tensor, w: torch.Tensor, counts: torch.Tensor,
                     out: torch.Tensor | None = None,
                     stream: torch.cuda.Stream | None = None) -> torch.Tensor:
    """dx [rows, k]: each expert's rows of dy [rows, n] times W_e, w [groups, n, k].  Rows
    behind the last expert's as in grouped_mm."""
    dev, rows, n, dt = rows_of("dy", dy)
    g, wn, k = _weights(w, dev, dt)
    if wn != n:
        raise ValueError(f"dy is {n} wide, w gives {wn}")
    check_tensor("counts", counts, dev, (g,), torch.int32)
    if out is not None:
        check_tensor("out", out, dev, (rows, k), dt)
    with on_stream(dev, stream, (dy, w, counts, out)) as s:
        if out is None:
            out = torch.empty(rows, k, dtype=dt, device=dev)
        check(lib().moe_grouped_mm_dgrad(dy.data_ptr(), w.data_ptr(), counts.data_ptr(), g, rows, n, k,
                                         DTYPES[dt], out.data_ptr(), s))
    return out


def grouped_mm_wgrad(dy: torch.Tensor, x: torch.Tensor, counts: torch.Tensor,
                     out: torch.Tensor | None = None, accumulate: bool = False,
                     stream: torch.cuda.Stream | None = None) -> torch.Tensor:
    """dW [groups, n, k] fp32: dy_e^T x_e over each expert's rows of dy [rows, n] and x [rows, k]
    (zeros for an expert without rows); with accumulate=True added to `out`."""
    dev, rows, n, dt = rows_of("dy", dy)
    xdev, xrows, k, xdt = rows_of("x", x)
    if (xdev, xrows, xdt) != (dev, rows, dt):
        raise ValueError("x and dy must have the same rows, type and device")
    if not isinstance(counts, torch.Tensor) or counts.dim() != 1:
        raise ValueError("counts must be a [groups] tensor")
    g = counts.shape[0]
    check_tensor("counts", counts, dev, (g,), torch.int32)
    if out is not None:
        check_tensor("out", out, dev, (g, n, k), torch.float32)
    elif accumulate:
        raise ValueError("accumulate=True adds to out: give it")
    with on_stream(dev, stream, (dy, x, counts, out)) as s:
        if out is None:
            out = torch.empty(g, n, k, dtype=torch.float32, device=dev)
        L = lib()
        size = L.moe_grouped_wgrad_workspace(g, rows, n, k, DTYPES[dt])
        ws = torch.empty(size, dtype=torch.uint8, device=dev) if size else None
        check(L.moe_grouped_mm_wgrad(dy.data_ptr(), x.data_ptr(), counts.data_ptr(), g, rows, n, k, DTYPES[dt],
                                     int(bool(accumulate)), out.data_ptr(), ws.data_ptr() if size else None,
                                     size, s))
    return out


def device_status(device=None, stream: torch.cuda.Stream | None = None) -> None:
    """Synchronise `stream` (default: the current stream of `device`) and raise if a grouped
    product on that device recorded a device-side error."""
    dev = torch.device("cuda" if device is None else device)
    if dev.index is None:
        dev = torch.device("cuda", torch.cuda.current_device())
    with on_stream(dev, stream) as s:
        check(lib().moe_grouped_device_status(s))
