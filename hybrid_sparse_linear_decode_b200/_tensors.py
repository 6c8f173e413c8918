"""Checks of tensor arguments, streams and devices for the calls that take tensors.

A decode step makes a few of these calls per layer, so what runs every time reads each attribute once and builds no
text; the messages are made when a check has failed.
"""

from __future__ import annotations

import torch

raw_stream = torch._C._cuda_getCurrentRawStream
current_device = torch._C._cuda_getDevice


def need(ok: bool, what: str) -> None:
    if not ok:
        raise ValueError(what)


def rows_of(t: torch.Tensor, name: str, heads: int, d: int, index: int, dtype=None) -> int:
    """Checks token rows [rows, heads, d] on device `index` whose heads are contiguous; returns the elements from row to row."""
    shape, stride = t.shape, t.stride()
    if (len(shape) != 3 or shape[1] != heads or shape[2] != d or t.get_device() != index or stride[2] != 1
            or (stride[1] != d and heads != 1) or (dtype is not None and t.dtype is not dtype)):
        need(t.get_device() == index, f"{name} is on {t.device}, not cuda:{index}")
        need(dtype is None or t.dtype is dtype, f"{name} is {t.dtype}, not {dtype}")
        need(len(shape) == 3 and shape[1] == heads and shape[2] == d, f"{name} has shape {list(shape)}, not [rows, {heads}, {d}]")
        raise ValueError(f"{name}: the heads of a row have to be contiguous (strides {list(stride)})")
    return stride[0] if shape[0] > 1 else heads * d


def vector_of(t: torch.Tensor, name: str, dtype, n: int, index: int) -> int:
    """Checks a contiguous vector of n elements; returns its address."""
    if t.dtype is not dtype or t.dim() != 1 or t.shape[0] != n or t.get_device() != index or not t.is_contiguous():
        raise ValueError(f"{name} has to be a contiguous {dtype} tensor of {n} elements on cuda:{index}, "
                         f"not {t.dtype} {list(t.shape)} on {t.device}")
    return t.data_ptr()


def run_on(index: int, stream, call):
    """Runs call(stream handle) with device `index` current, on the caller's stream if one is given, so that what the
    call allocates belongs to the stream that uses it."""
    if stream is None:
        if current_device() == index:
            return call(raw_stream(index))
        with torch.cuda.device(index):
            return call(raw_stream(index))
    if not isinstance(stream, torch.cuda.Stream):
        stream = torch.cuda.ExternalStream(int(stream), device=torch.device("cuda", index))
    with torch.cuda.stream(stream):
        return call(stream.cuda_stream)
