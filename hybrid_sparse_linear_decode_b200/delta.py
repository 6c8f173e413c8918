"""The states of one gated-delta-rule layer, and the call that takes tokens through them.

PyTorch is used for device memory and streams only; the work is the library's.
"""

from __future__ import annotations

import torch

from . import _abi as A
from ._tensors import need, rows_of, run_on, vector_of


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

    def run(self, q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, g: torch.Tensor, beta: torch.Tensor, cu: torch.Tensor,
            max_new: int, slots: torch.Tensor | None = None, scale: float = 0.0, out: torch.Tensor | None = None,
            stream=None) -> torch.Tensor:
        """Takes a step's tokens through the states in place.  Sequence b owns rows cu[b] .. cu[b + 1] (int32, device) and
        state ``slots[b]`` (int32, device; default b; -1: the sequence is skipped, its rows stay as they were); ``max_new``
        bounds the rows of one sequence.  q, k [rows, n_k_heads, key_dim], v [rows, n_v_heads, value_dim] bf16; g, beta
        [rows, n_v_heads] fp32.  Returns [rows, n_v_heads, value_dim] bf16."""
        index, dtype = self._index, torch.bfloat16
        Hv, dv = self.n_v_heads, self.value_dim
        qs = rows_of(q, "q", self.n_k_heads, self.key_dim, index, dtype)
        ks = rows_of(k, "k", self.n_k_heads, self.key_dim, index, dtype)
        vs = rows_of(v, "v", Hv, dv, index, dtype)
        n = q.shape[0]
        need(k.shape[0] == n and v.shape[0] == n, "q, k and v have as many rows")
        for t, name in ((g, "g"), (beta, "beta")):
            if t.dtype is not torch.float32 or t.shape != (n, Hv) or t.get_device() != index or not t.is_contiguous():
                raise ValueError(f"{name} has to be a contiguous fp32 [{n}, {Hv}] tensor on {self.device}")
        need(cu.dim() == 1 and cu.shape[0] >= 2, "cu is [B + 1]")
        B = cu.shape[0] - 1
        need(max_new >= 1 or n == 0, "max_new is at least 1")
        cu_at = vector_of(cu, "cu", torch.int32, B + 1, index)
        slots_at = None if slots is None else vector_of(slots, "slots", torch.int32, B, index)
        os = Hv * dv
        if out is not None:
            os = rows_of(out, "out", Hv, dv, index, dtype)
            need(out.shape[0] == n, "out has as many rows as q")

        def call(handle):
            to = q.new_empty((n, Hv, dv)) if out is None else out
            A.hyb_attn_delta_run(self._c, q.data_ptr(), qs, k.data_ptr(), ks, v.data_ptr(), vs, g.data_ptr(), beta.data_ptr(),
                                 to.data_ptr(), os, cu_at, slots_at, B, n, max_new if max_new < n else n, scale,
                                 self._status_at, handle)
            return to

        return run_on(index, stream, call)

    def status(self, clear: bool = False) -> int:
        """The HYB_STATUS_* bits raised by these states' calls so far (waits for them)."""
        flags = int(self._status.item())
        if clear:
            self._status.zero_()
        return flags
