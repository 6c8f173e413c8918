"""The states of one gated-delta-rule layer, and the call that takes tokens through them.

PyTorch is used for device memory and streams only; the work is the library's.
"""

from __future__ import annotations

import ctypes

import torch

from . import _abi as A
from ._tensors import binding, need, on_stream, read_status


class GatedDeltaState:
    """fp32 states ``state`` [n_slots, n_v_heads, key_dim, value_dim]; a sequence keeps one slot.

    For each token, with a = exp(g): S := a S; S := S + k (beta (v - S^T k))^T; o = scale S^T q.  Head i of v, g, beta
    and the output uses head i // (n_v_heads // n_k_heads) of q and k.
    """

    def __init__(self, n_slots: int, n_k_heads: int, n_v_heads: int, key_dim: int, value_dim: int, device=None):
        if not torch.cuda.is_available():
            raise RuntimeError("GatedDeltaState needs a CUDA device (sm_100a); there is no CPU path")
        self._bind(torch.zeros((n_slots, n_v_heads, key_dim, value_dim), dtype=torch.float32,
                               device=device if device is not None else "cuda"), n_k_heads)

    @classmethod
    def from_tensor(cls, state: torch.Tensor, n_k_heads: int) -> "GatedDeltaState":
        """States in the caller's own tensor."""
        self = cls.__new__(cls)
        self._bind(state, n_k_heads)
        return self

    def _bind(self, state, n_k_heads) -> None:
        need(state.dim() == 4 and state.dtype == torch.float32 and state.is_contiguous(),
             "the states are a contiguous fp32 [n_slots, n_v_heads, key_dim, value_dim] tensor")
        need(state.is_cuda, "the states are on a CUDA device; there is no CPU path")
        self.state, self.n_k_heads = state, n_k_heads
        self.n_slots, self.n_v_heads, self.key_dim, self.value_dim = state.shape
        self.device = state.device
        self._index = state.get_device()
        self._status = torch.zeros(1, dtype=torch.int32, device=state.device)
        self._status_at = self._status.data_ptr()
        self._c = A.hyb_attn_delta_state(state.data_ptr(), self.n_slots, n_k_heads, self.n_v_heads, self.key_dim, self.value_dim)
        self._c_at = ctypes.addressof(self._c)
        self._calls = binding()

    def run(self, q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, g: torch.Tensor, beta: torch.Tensor, cu: torch.Tensor,
            max_new: int, slots: torch.Tensor | None = None, scale: float = 0.0, out: torch.Tensor | None = None,
            stream=None) -> torch.Tensor:
        """Takes a step's tokens through the states in place.  Sequence b owns rows cu[b] .. cu[b + 1] (int32, device) and
        state ``slots[b]`` (int32, device; default b; -1: the sequence is skipped, its rows stay as they were); ``max_new``
        bounds the rows of one sequence.  q, k [rows, n_k_heads, key_dim], v [rows, n_v_heads, value_dim] bf16; g, beta
        [rows, n_v_heads] fp32.  Returns [rows, n_v_heads, value_dim] bf16 (``out``, if given, in other memory than the
        inputs).  Tokens cannot be taken out of a state again: for drafts that may be rejected keep a copy of it."""
        if stream is not None:
            with on_stream(stream, self.device):
                return self.run(q, k, v, g, beta, cu, max_new, slots, scale, out)
        return self._calls.delta_run(self._c_at, self._index, self._status_at, q, k, v, g, beta, cu, max_new, slots, scale, out)

    def status(self, clear: bool = False) -> int:
        """The HYB_STATUS_* bits raised by these states' calls so far, on whatever stream (waits for the device)."""
        return read_status(self._status, clear)
