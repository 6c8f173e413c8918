"""One layer's paged cache of 8-bit codes, and the calls that append to it and attend over it.

PyTorch is used for device memory and streams only; the work is the library's.
"""

from __future__ import annotations

import contextlib

import torch

from . import _abi as A

_CODES = {torch.float8_e4m3fn: A.HYB_CODE_E4M3, torch.int8: A.HYB_CODE_INT8}
_TYPES = {torch.bfloat16: A.HYB_TYPE_BF16, torch.float16: A.HYB_TYPE_FP16}


def need(ok: bool, what: str) -> None:
    if not ok:
        raise ValueError(what)


def on_device(device: torch.device, stream):
    """The context that a call runs in: its tensors' device, and the caller's stream if one is given, so that what the
    call allocates belongs to the stream that uses it."""
    if stream is None:
        if device.index == torch.cuda.current_device():
            return contextlib.nullcontext()
        return torch.cuda.device(device)
    if not isinstance(stream, torch.cuda.Stream):
        stream = torch.cuda.ExternalStream(int(stream), device=device)
    return torch.cuda.stream(stream)


def heads_of(t: torch.Tensor, name: str, n: int, d: int, device, dtype=None) -> int:
    """Checks token rows [n_new][heads][d] whose heads are contiguous; returns the elements from row to row."""
    need(t.dim() == 3 and t.shape[1] == n and t.shape[2] == d, f"{name} has shape {tuple(t.shape)}, not [rows, {n}, {d}]")
    need(t.device == device, f"{name} is on {t.device}, the state on {device}")
    need(dtype is None or t.dtype == dtype, f"{name} is {t.dtype}, not {dtype}")
    need(t.stride(2) == 1 and (n == 1 or t.stride(1) == d), f"{name}: the heads of a row have to be contiguous")
    return t.stride(0) if t.shape[0] > 1 else max(t.stride(0), n * d)


def ints_of(t: torch.Tensor, name: str, device, *shape) -> int:
    need(t.dtype == torch.int32 and t.device == device and t.is_contiguous() and t.shape == shape,
         f"{name} has to be a contiguous int32 tensor of shape {list(shape)} on {device}")
    return t.data_ptr()


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
        self._status = torch.zeros(1, dtype=torch.int32, device=k.device)
        self._c = A.hyb_attn_paged_cache(k.data_ptr(), v.data_ptr(), ks.data_ptr(), vs.data_ptr(), *k.shape, _CODES[k.dtype])

    def _batch(self, cu, kv_lens, page_table, n_new, max_new, max_len) -> A.hyb_attn_paged_batch:
        need(page_table.dim() == 2, "page_table is [B, pages]")
        B, pages = page_table.shape
        dev = self.device
        return A.hyb_attn_paged_batch(ints_of(page_table, "page_table", dev, B, pages), ints_of(cu, "cu", dev, B + 1),
                                      ints_of(kv_lens, "kv_lens", dev, B), B, pages, n_new, min(int(max_new), n_new),
                                      max_len, self._status.data_ptr())

    def append(self, k: torch.Tensor, v: torch.Tensor, cu: torch.Tensor, kv_lens: torch.Tensor, page_table: torch.Tensor,
               max_new: int, rope: torch.Tensor | None = None, interleaved: bool = False, q: torch.Tensor | None = None,
               q_out: torch.Tensor | None = None, stream=None) -> torch.Tensor | None:
        """Append a step's tokens: k, v [rows, n_kv_heads, d] (bf16 or fp16), keys rotated by ``rope`` (fp32
        [positions, rot_dim]: cosines, then sines).  With ``q`` [rows, n_q_heads, d] returns the queries rotated alike
        (into ``q_out``, which may be ``q``)."""
        n, d = k.shape[0], self.head_dim
        need(k.dtype in _TYPES, f"k is {k.dtype}, not bfloat16 or float16")
        ks = heads_of(k, "k", self.n_kv_heads, d, self.device)
        vs = heads_of(v, "v", self.n_kv_heads, d, self.device, k.dtype)
        need(v.shape[0] == n, "k and v have as many rows")
        need(max_new >= 1 or n == 0, "max_new is at least 1")
        n_pos = rot = 0
        if rope is not None:
            need(rope.dim() == 2 and rope.dtype == torch.float32 and rope.is_contiguous() and rope.device == self.device,
                 "rope is a contiguous fp32 [positions, rot_dim] tensor on the cache's device")
            n_pos, rot = rope.shape
        b = self._batch(cu, kv_lens, page_table, n, max_new, 0)
        with on_device(self.device, stream):
            heads = qs = qo = 0
            if q is not None:
                need(q.dim() == 3 and q.shape[0] == n, "q has as many rows as k")
                heads = q.shape[1]
                qs = heads_of(q, "q", heads, d, self.device, k.dtype)
                if q_out is None:
                    q_out = torch.empty((n, heads, d), dtype=q.dtype, device=self.device)
                qo = heads_of(q_out, "q_out", heads, d, self.device, k.dtype)
                need(q_out.shape[0] == n, "q_out has as many rows as q")
            else:
                need(q_out is None, "q_out without q")
            A.hyb_attn_paged_append(self._c, b, _TYPES[k.dtype], k.data_ptr(), ks, v.data_ptr(), vs,
                                    None if rope is None else rope.data_ptr(), n_pos, rot, interleaved,
                                    None if q is None else q.data_ptr(), qs,
                                    None if q is None else q_out.data_ptr(), qo, heads,
                                    torch.cuda.current_stream().cuda_stream)
        return q_out

    def attend(self, q: torch.Tensor, cu: torch.Tensor, kv_lens: torch.Tensor, page_table: torch.Tensor, max_new: int,
               max_len: int, window: int = 0, n_sink: int = 0, scale: float = 0.0, out: torch.Tensor | None = None,
               return_lse: bool = False, stream=None):
        """Causal attention of the step's tokens q [rows, n_q_heads, d] over the cache (append them first): returns out
        [rows, n_q_heads, d] in q's type, with ``return_lse`` also the fp32 [rows, n_q_heads] logarithms of the softmax
        sums.  ``window`` > 0 hides positions t - window and before, but for the first ``n_sink``.  Rows behind
        the last sequence are left as they were (in new tensors: not written)."""
        need(q.dim() == 3 and q.dtype in _TYPES, "q is [rows, n_q_heads, head_dim], bfloat16 or float16")
        n, heads, d = q.shape
        qs = heads_of(q, "q", heads, self.head_dim, self.device)
        need(max_new >= 1 or n == 0, "max_new is at least 1")
        b = self._batch(cu, kv_lens, page_table, n, max_new, max_len)
        with on_device(self.device, stream):
            if out is None:
                out = torch.empty((n, heads, d), dtype=q.dtype, device=self.device)
            os = heads_of(out, "out", heads, d, self.device, q.dtype)
            need(out.shape[0] == n, "out has as many rows as q")
            lse = torch.empty((n, heads), dtype=torch.float32, device=self.device) if return_lse else None
            size = A.hyb_attn_paged_workspace_size(self._c, b, heads)
            ws = torch.empty(size, dtype=torch.uint8, device=self.device) if size else None
            A.hyb_attn_paged_attend(self._c, b, _TYPES[q.dtype], q.data_ptr(), qs, out.data_ptr(), os,
                                    lse.data_ptr() if return_lse else None, heads, window, n_sink, scale,
                                    ws.data_ptr() if size else None, size, torch.cuda.current_stream().cuda_stream)
        return (out, lse) if return_lse else out

    def status(self, clear: bool = False) -> int:
        """The HYB_STATUS_* bits raised by this cache's calls so far (waits for them)."""
        flags = int(self._status.item())
        if clear:
            self._status.zero_()
        return flags
