"""What the classes over PyTorch tensors share: checks, the compiled calls and the caller's stream."""

from __future__ import annotations

import torch

from . import _abi as A


def need(ok: bool, what: str) -> None:
    if not ok:
        raise ValueError(what)


def binding():
    """The compiled calls (``_binding.so``, built with the library); a missing one is an error, there is no fallback."""
    A.load_library()
    try:
        from . import _binding
    except ImportError as e:
        raise RuntimeError("_binding.so is missing or does not load: build it with "
                           "`python -m hybrid_sparse_linear_decode_b200.build`") from e
    return _binding


def read_status(word: torch.Tensor, clear: bool) -> int:
    """A handle's status word once all work on its device is done: its calls may have been made, or replayed, on any stream."""
    torch.cuda.synchronize(word.device)
    flags = int(word.item())
    if clear:
        word.zero_()
        torch.cuda.synchronize(word.device)  # before whatever another stream raises next
    return flags


def on_stream(stream, device: torch.device):
    """The caller's stream as the current one, so that what a call allocates belongs to the stream that uses it."""
    if not isinstance(stream, torch.cuda.Stream):
        stream = torch.cuda.ExternalStream(int(stream), device=device)
    need(stream.device == device, f"the stream belongs to {stream.device}, the buffers to {device}")
    return torch.cuda.stream(stream)
