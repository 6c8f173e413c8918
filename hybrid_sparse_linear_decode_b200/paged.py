"""One layer's paged cache of 8-bit codes, and the calls that append to it and attend over it.

PyTorch is used for device memory and streams only; the work is the library's.
"""

from __future__ import annotations

import ctypes

import torch

from . import _abi as A
from ._tensors import binding, need, on_stream, read_status

_CODES = {torch.float8_e4m3fn: A.HYB_CODE_E4M3, torch.int8: A.HYB_CODE_INT8}


class PagedKVCache:
    """Codes ``[n_pages, n_kv_heads, page_size, head_dim]`` (float8_e4m3fn or int8) and scales
    ``[n_pages, n_kv_heads]`` (fp32) of keys and values: ``k_pages, v_pages, k_scales, v_scales``.

    A step's sequences are given by three int32 device tensors: ``cu`` [B + 1] (sequence b owns token rows
    cu[b] .. cu[b + 1]), ``kv_lens`` [B] (its tokens once the new ones are counted) and ``page_table`` [B, pages].
    ``max_new`` and ``max_len`` bound a sequence's new tokens and tokens in all.  Rows past ``max_new`` and tokens at
    positions or on pages that the table or the cache does not have are skipped, and noted in ``status``; the others keep
    their positions.
    """

    def __init__(self, n_pages: int, page_size: int, n_kv_heads: int, head_dim: int, dtype=torch.float8_e4m3fn,
                 device=None):
        if not torch.cuda.is_available():
            raise RuntimeError("PagedKVCache needs a CUDA device (sm_100a); there is no CPU path")
        need(dtype in _CODES, f"codes are float8_e4m3fn or int8, not {dtype}")
        dev = torch.device(device if device is not None else "cuda")
        shape = (n_pages, n_kv_heads, page_size, head_dim)
        k, v = (torch.zeros(shape, dtype=torch.int8, device=dev).view(dtype) for _ in "kv")
        ks, vs = (torch.zeros(shape[:2], dtype=torch.float32, device=dev) for _ in "kv")
        self._bind(k, v, ks, vs)

    @classmethod
    def from_tensors(cls, k_pages: torch.Tensor, v_pages: torch.Tensor, k_scales: torch.Tensor,
                     v_scales: torch.Tensor) -> "PagedKVCache":
        """A cache over the caller's own tensors."""
        self = cls.__new__(cls)
        self._bind(k_pages, v_pages, k_scales, v_scales)
        return self

    def _bind(self, k, v, ks, vs) -> None:
        need(k.dim() == 4 and k.dtype in _CODES, "codes are [n_pages, n_kv_heads, page_size, head_dim], float8_e4m3fn or int8")
        for t in (v, ks, vs):
            need(t.device == k.device, "codes and scales are on one device")
        need(v.dtype == k.dtype and v.shape == k.shape, "keys and values have codes of one shape and type")
        need(all(t.dtype == torch.float32 and t.shape == k.shape[:2] for t in (ks, vs)), "scales are fp32 [n_pages, n_kv_heads]")
        need(all(t.is_contiguous() for t in (k, v, ks, vs)), "codes and scales are contiguous")
        need(k.is_cuda, "the cache is on a CUDA device; there is no CPU path")
        self.k_pages, self.v_pages, self.k_scales, self.v_scales = k, v, ks, vs
        self.n_pages, self.n_kv_heads, self.page_size, self.head_dim = k.shape
        self.device = k.device
        self._index = k.get_device()
        self._status = torch.zeros(1, dtype=torch.int32, device=k.device)
        self._status_at = self._status.data_ptr()
        self._c = A.hyb_attn_paged_cache(k.data_ptr(), v.data_ptr(), ks.data_ptr(), vs.data_ptr(), *k.shape, _CODES[k.dtype])
        self._c_at = ctypes.addressof(self._c)
        self._calls = binding()

    def append(self, k: torch.Tensor, v: torch.Tensor, cu: torch.Tensor, kv_lens: torch.Tensor, page_table: torch.Tensor,
               max_new: int, rope: torch.Tensor | None = None, interleaved: bool = False, q: torch.Tensor | None = None,
               q_out: torch.Tensor | None = None, stream=None) -> torch.Tensor | None:
        """Append a step's tokens: k, v [rows, n_kv_heads, d] (bf16 or fp16), keys rotated by ``rope`` (fp32
        [positions, rot_dim]: cosines, then sines).  With ``q`` [rows, n_q_heads, d] returns the queries rotated alike
        (into ``q_out``, which may be ``q``).  ``stream``: the caller's stream instead of the current one; tensors made on
        another one have to outlive the call (``record_stream``)."""
        if stream is not None:
            with on_stream(stream, self.device):
                return self.append(k, v, cu, kv_lens, page_table, max_new, rope, interleaved, q, q_out)
        return self._calls.paged_append(self._c_at, self._index, self._status_at, k, v, cu, kv_lens, page_table, max_new, rope,
                                        interleaved, q, q_out)

    def attend(self, q: torch.Tensor, cu: torch.Tensor, kv_lens: torch.Tensor, page_table: torch.Tensor, max_new: int,
               max_len: int, window: int = 0, n_sink: int = 0, scale: float = 0.0, out: torch.Tensor | None = None,
               return_lse: bool = False, stream=None):
        """Causal attention of the step's tokens q [rows, n_q_heads, d] over the cache (append them first): returns out
        [rows, n_q_heads, d] in q's type, with ``return_lse`` also the fp32 [rows, n_q_heads] logarithms of the softmax
        sums.  ``window`` > 0 hides positions t - window and before, but for the first ``n_sink``.  Rows behind
        the last sequence are left as they were (in new tensors: not written).  ``out`` is in other memory than q;
        ``scale`` 0 selects 1/sqrt(d)."""
        if stream is not None:
            with on_stream(stream, self.device):
                return self.attend(q, cu, kv_lens, page_table, max_new, max_len, window, n_sink, scale, out, return_lse)
        return self._calls.paged_attend(self._c_at, self._index, self._status_at, q, cu, kv_lens, page_table, max_new, max_len,
                                        window, n_sink, scale, out, return_lse)

    def status(self, clear: bool = False) -> int:
        """The HYB_STATUS_* bits raised by this cache's calls so far, on whatever stream (waits for the device)."""
        return read_status(self._status, clear)
