"""One layer's paged cache of 8-bit codes, and the calls that append to it and attend over it.

PyTorch is used for device memory and streams only; the work is the library's.
"""

from __future__ import annotations

import torch

from . import _abi as A
from ._tensors import need, rows_of, run_on, vector_of

_CODES = {torch.float8_e4m3fn: A.HYB_CODE_E4M3, torch.int8: A.HYB_CODE_INT8}
_TYPES = {torch.bfloat16: A.HYB_TYPE_BF16, torch.float16: A.HYB_TYPE_FP16}


class PagedKVCache:
    """Codes ``[n_pages, n_kv_heads, page_size, head_dim]`` (float8_e4m3fn or int8) and scales
    ``[n_pages, n_kv_heads]`` (fp32) of keys and values: ``k_pages, v_pages, k_scales, v_scales``.

    A step's sequences are given by three int32 device tensors: ``cu`` [B + 1] (sequence b owns token rows
    cu[b] .. cu[b + 1]), ``kv_lens`` [B] (its tokens once the new ones are counted) and ``page_table`` [B, pages].
    ``max_new`` and ``max_len`` bound a sequence's new tokens and tokens in all.  What contradicts the bounds or the
    table is held to them or skipped, and noted in ``status``.
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
        self._sizes = {}  # workspace bytes by the limits that they follow from
        self._c = A.hyb_attn_paged_cache(k.data_ptr(), v.data_ptr(), ks.data_ptr(), vs.data_ptr(), *k.shape, _CODES[k.dtype])

    def _batch(self, cu, kv_lens, page_table, n_new, max_new, max_len) -> A.hyb_attn_paged_batch:
        index = self._index
        if (page_table.dtype is not torch.int32 or page_table.dim() != 2 or page_table.get_device() != index
                or not page_table.is_contiguous()):
            raise ValueError(f"page_table has to be a contiguous int32 [B, pages] tensor on {self.device}")
        B, pages = page_table.shape
        need(max_new >= 1 or n_new == 0, "max_new is at least 1")
        return A.hyb_attn_paged_batch(page_table.data_ptr(), vector_of(cu, "cu", torch.int32, B + 1, index),
                                      vector_of(kv_lens, "kv_lens", torch.int32, B, index), B, pages, n_new,
                                      max_new if max_new < n_new else n_new, max_len, self._status_at)

    def append(self, k: torch.Tensor, v: torch.Tensor, cu: torch.Tensor, kv_lens: torch.Tensor, page_table: torch.Tensor,
               max_new: int, rope: torch.Tensor | None = None, interleaved: bool = False, q: torch.Tensor | None = None,
               q_out: torch.Tensor | None = None, stream=None) -> torch.Tensor | None:
        """Append a step's tokens: k, v [rows, n_kv_heads, d] (bf16 or fp16), keys rotated by ``rope`` (fp32
        [positions, rot_dim]: cosines, then sines).  With ``q`` [rows, n_q_heads, d] returns the queries rotated alike
        (into ``q_out``, which may be ``q``)."""
        index, d, dtype = self._index, self.head_dim, k.dtype
        if dtype not in _TYPES:
            raise ValueError(f"k is {dtype}, not bfloat16 or float16")
        ks = rows_of(k, "k", self.n_kv_heads, d, index)
        vs = rows_of(v, "v", self.n_kv_heads, d, index, dtype)
        n = k.shape[0]
        need(v.shape[0] == n, "k and v have as many rows")
        n_pos = rot = heads = qs = qo = 0
        rope_at = q_at = qo_at = None
        if rope is not None:
            if rope.dim() != 2 or rope.dtype is not torch.float32 or rope.get_device() != index or not rope.is_contiguous():
                raise ValueError("rope has to be a contiguous fp32 [positions, rot_dim] tensor on the cache's device")
            n_pos, rot = rope.shape
            rope_at = rope.data_ptr()
        if q is not None:
            need(q.dim() == 3 and q.shape[0] == n, "q is [rows, n_q_heads, head_dim], with as many rows as k")
            heads, q_at = q.shape[1], q.data_ptr()
            qs = rows_of(q, "q", heads, d, index, dtype)
            if q_out is not None:
                qo, qo_at = rows_of(q_out, "q_out", heads, d, index, dtype), q_out.data_ptr()
                need(q_out.shape[0] == n, "q_out has as many rows as q")
        else:
            need(q_out is None, "q_out without q")
        b = self._batch(cu, kv_lens, page_table, n, max_new, 0)

        def call(handle):
            to, to_at, to_stride = q_out, qo_at, qo
            if q is not None and to is None:
                to = q.new_empty((n, heads, d))
                to_at, to_stride = to.data_ptr(), heads * d
            A.hyb_attn_paged_append(self._c, b, _TYPES[dtype], k.data_ptr(), ks, v.data_ptr(), vs, rope_at, n_pos, rot,
                                    interleaved, q_at, qs, to_at, to_stride, heads, handle)
            return to

        return run_on(index, stream, call)

    def attend(self, q: torch.Tensor, cu: torch.Tensor, kv_lens: torch.Tensor, page_table: torch.Tensor, max_new: int,
               max_len: int, window: int = 0, n_sink: int = 0, scale: float = 0.0, out: torch.Tensor | None = None,
               return_lse: bool = False, stream=None):
        """Causal attention of the step's tokens q [rows, n_q_heads, d] over the cache (append them first): returns out
        [rows, n_q_heads, d] in q's type, with ``return_lse`` also the fp32 [rows, n_q_heads] logarithms of the softmax
        sums.  ``window`` > 0 hides positions t - window and before, but for the first ``n_sink``.  Rows behind
        the last sequence are left as they were (in new tensors: not written)."""
        index, d, dtype = self._index, self.head_dim, q.dtype
        if dtype not in _TYPES or q.dim() != 3:
            raise ValueError("q has to be [rows, n_q_heads, head_dim], bfloat16 or float16")
        n, heads, _ = q.shape
        qs = rows_of(q, "q", heads, d, index)
        b = self._batch(cu, kv_lens, page_table, n, max_new, max_len)
        key = (n, heads, b.max_new, max_len, b.batch, b.table_stride)
        size = self._sizes.get(key)
        if size is None:
            if len(self._sizes) > 256:
                self._sizes.clear()
            size = self._sizes[key] = A.hyb_attn_paged_workspace_size(self._c, b, heads)
        os = heads * d
        if out is not None:
            os = rows_of(out, "out", heads, d, index, dtype)
            need(out.shape[0] == n, "out has as many rows as q")

        def call(handle):
            to = q.new_empty((n, heads, d)) if out is None else out
            lse = q.new_empty((n, heads), dtype=torch.float32) if return_lse else None
            ws = q.new_empty(size, dtype=torch.uint8) if size else None
            A.hyb_attn_paged_attend(self._c, b, _TYPES[dtype], q.data_ptr(), qs, to.data_ptr(), os,
                                    lse.data_ptr() if return_lse else None, heads, window, n_sink, scale,
                                    ws.data_ptr() if size else None, size, handle)
            return (to, lse) if return_lse else to

        return run_on(index, stream, call)

    def status(self, clear: bool = False) -> int:
        """The HYB_STATUS_* bits raised by this cache's calls so far (waits for them)."""
        flags = int(self._status.item())
        if clear:
            self._status.zero_()
        return flags
