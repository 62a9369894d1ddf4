"""Paged key/value cache of an ordinary attention layer (separate keys and values, H query heads on
H_kv key/value heads): the local and full-attention layers beside a model's compressed ones.

  pools   k_pages, v_pages : [num_pages, page_size, H_kv, d] bf16 or fp16, any order of the first three
                             dimensions in memory (a [num_pages, H_kv, page_size, d] pool is passed as
                             its transpose(1, 2))
  table   page_table       : [B, max_pages] int32, the page of tokens [j page_size, (j + 1) page_size)
  table   seqs             : [B, 3] int64 = (row, n, len) = csa_kv_seq: sequence b holds len tokens, the
                             newest n of them are rows [row, row + n) of the token arrays

The tensors stay the caller's: PagedKV checks them once and fills the C structs.  The ``*_args`` methods
return the arguments of one call, which can be used again as long as the tensors in them live (they are
kept alive by the arguments, and go with them: on a stream other than the tensors' own, drop the
arguments only after the call's work is done); the tables' contents may change between calls, also between
replays of a captured graph.  ``append`` writes new tokens (turning keys and queries by position), ``window_attn`` and
``prefix_attn`` attend them.  Calls run on the current stream of the cache's device unless given one.
Torch is used for allocation and checks only.
"""
from __future__ import annotations

from ctypes import byref

from . import (CSA_KV_BF16, CSA_KV_F16, CSA_OP_PREFIX_ATTN, CSA_OP_WINDOW_ATTN, _check, csa_kv_append_args,
               csa_kv_attn_args, csa_kv_cache, csa_workspace_size, lib)


def _need(ok, what):
    if not ok:
        raise ValueError(what)


class PagedKV:
    """k_pages / v_pages / page_table / seqs as above; H: query heads (a multiple of H_kv)."""

    def __init__(self, k_pages, v_pages, page_table, seqs, H):
        import torch

        _need(k_pages.dim() == 4 and v_pages.shape == k_pages.shape, "k_pages and v_pages are [num_pages, page_size, H_kv, d]")
        _need(k_pages.dtype == v_pages.dtype and k_pages.dtype in (torch.bfloat16, torch.float16),
              f"pages of {k_pages.dtype} / {v_pages.dtype}: bfloat16 or float16")
        _need(v_pages.stride() == k_pages.stride() and (k_pages.stride(3) == 1 or k_pages.shape[3] == 1),
              "the pools need the same strides and contiguous channels")
        _need(page_table.dtype == torch.int32 and page_table.dim() == 2 and page_table.is_contiguous(),
              "page_table is a contiguous [B, max_pages] int32 tensor")
        _need(seqs.dtype == torch.int64 and seqs.shape == (page_table.shape[0], 3) and seqs.is_contiguous(),
              "seqs is a contiguous [B, 3] int64 tensor")
        self.device = k_pages.device
        _need(self.device.type == "cuda", f"pages on {self.device}")
        for t in (v_pages, page_table, seqs):
            _need(t.device == self.device, f"tensors on {t.device} and {self.device}")
        self.k_pages, self.v_pages, self.page_table, self.seqs = k_pages, v_pages, page_table, seqs
        num_pages, page, H_kv, d = k_pages.shape
        self.H, self.H_kv, self.d, self.dtype = int(H), H_kv, d, k_pages.dtype
        kv = self.kv = csa_kv_cache()
        kv.H, kv.H_kv, kv.d, kv.page_size, kv.B = self.H, H_kv, d, page, page_table.shape[0]
        kv.type = CSA_KV_F16 if self.dtype == torch.float16 else CSA_KV_BF16
        kv.num_pages, kv.max_pages = num_pages, page_table.shape[1]
        kv.page_stride, kv.slot_stride, kv.head_stride = k_pages.stride()[:3]
        kv.k_pages, kv.v_pages = k_pages.data_ptr(), v_pages.data_ptr()
        kv.page_table, kv.seqs = page_table.data_ptr(), seqs.data_ptr()
        # a call costs the host a few microseconds: what it needs is looked up here
        self._device_index = self.device.index
        self._current_stream, self._current_device = torch._C._cuda_getCurrentRawStream, torch._C._cuda_getDevice
        so = lib()
        self._append_fn, self._window_fn, self._prefix_fn = so.csa_kv_append, so.csa_window_attn, so.csa_prefix_attn

    def _rows(self, t, heads, name):
        """Row stride of a [rows, heads, d] token array with contiguous heads."""
        _need(t.dim() == 3 and t.shape[1:] == (heads, self.d), f"{name} is [rows, {heads}, {self.d}], got {tuple(t.shape)}")
        _need(t.dtype == self.dtype and t.device == self.device, f"{name}: {t.dtype} on {t.device}, the cache is "
              f"{self.dtype} on {self.device}")
        _need(t.stride(2) == 1 and (heads == 1 or t.stride(1) == self.d), f"the heads of {name} must be contiguous")
        return t.stride(0) if t.shape[0] > 1 else heads * self.d

    def append_args(self, k, v, q=None, q_out=None, *, max_n, inv_freq=None, interleaved=False) -> csa_kv_append_args:
        """New tokens k, v [rows, H_kv, d]; optional queries q [rows, H, d] turned into q_out (q itself: in
        place).  inv_freq: float32 [rot / 2], the angle per position of each channel pair (None or
        empty: no rotation); max_n: bound of every sequence's n."""
        import torch

        a = csa_kv_append_args()
        a.kv, a.rows, a.max_n = self.kv, k.shape[0], int(max_n)
        a.k_stride, a.v_stride = self._rows(k, self.H_kv, "k"), self._rows(v, self.H_kv, "v")
        _need(v.shape[0] == k.shape[0], "k and v have different numbers of rows")
        a.k, a.v = k.data_ptr(), v.data_ptr()
        _need((q is None) == (q_out is None), "q and q_out go together")
        if q is not None:
            a.q_stride, a.q_out_stride = self._rows(q, self.H, "q"), self._rows(q_out, self.H, "q_out")
            _need(q.shape[0] == k.shape[0] and q_out.shape[0] == k.shape[0], "q, q_out and k have different numbers of rows")
            a.q, a.q_out = q.data_ptr(), q_out.data_ptr()
        if inv_freq is not None and inv_freq.numel():
            _need(inv_freq.dtype == torch.float32 and inv_freq.dim() == 1 and inv_freq.is_contiguous() and
                  inv_freq.device == self.device, "inv_freq is a contiguous float32 vector on the cache's device")
            a.inv_freq, a.rot = inv_freq.data_ptr(), 2 * inv_freq.numel()
        a.interleaved = 1 if interleaved else 0
        a._keep = (self, k, v, q, q_out, inv_freq)
        return a

    def _attn_args(self, q, out, max_n, max_len, lse, scale):
        import torch

        a = csa_kv_attn_args()
        a.kv, a.rows, a.max_n = self.kv, q.shape[0], int(max_n)
        a.max_len = int(max_len if max_len is not None else self.kv.max_pages * self.kv.page_size)
        a.scale = float(scale if scale is not None else self.d ** -0.5)
        a.q_stride, a.out_stride = self._rows(q, self.H, "q"), self._rows(out, self.H, "out")
        _need(out.shape[0] == q.shape[0], "q and out have different numbers of rows")
        a.q, a.out = q.data_ptr(), out.data_ptr()
        if lse is not None:
            _need(lse.dtype == torch.float32 and lse.shape == (q.shape[0], self.H) and lse.is_contiguous() and
                  lse.device == self.device, "lse is a contiguous float32 [rows, H] tensor on the cache's device")
            a.lse = lse.data_ptr()
        a._keep = (self, q, out, lse)
        return a

    def window_args(self, q, out, *, W, S=0, max_n, max_len=None, lse=None, scale=None) -> csa_kv_attn_args:
        """q, out [rows, H, d]: attention over each query's last W tokens (itself among them) and the
        first S of its sequence.  max_n, max_len: bounds of every sequence's n and len."""
        a = self._attn_args(q, out, max_n, max_len, lse, scale)
        a.W, a.S = int(W), int(S)
        a._op = CSA_OP_WINDOW_ATTN
        return a

    def prefix_args(self, q, out, *, prefix_len, max_n, max_len=None, lse=None, scale=None) -> csa_kv_attn_args:
        """q, out [rows, H, d]: causal attention of sequences that share their first prefix_len tokens
        (read through row 0 of the table)."""
        a = self._attn_args(q, out, max_n, max_len, lse, scale)
        a.prefix_len = int(prefix_len)
        a._op = CSA_OP_PREFIX_ATTN
        return a

    def workspace(self, args):
        """A workspace for one call with `args` (calls that may overlap need one each)."""
        import torch

        with torch.cuda.device(self.device):
            n = csa_workspace_size(args._op, args)
        if n == 0:  # refused: let the call name the reason
            n = 256
        return torch.empty(n, dtype=torch.uint8, device=self.device)

    def _call(self, name, fn, stream, *args):
        index = self._device_index
        if stream is None:
            stream = self._current_stream(index)
        elif not isinstance(stream, int):
            _need(stream.device == self.device, f"a stream of {stream.device} for a cache on {self.device}")
            stream = stream.cuda_stream
        if self._current_device() == index:
            rc = fn(*args, stream)
        else:
            import torch

            with torch.cuda.device(index):
                rc = fn(*args, stream)
        if rc:
            _check(rc, name)

    def _space(self, ws):
        if ws is None:
            return None, 0
        if ws.get_device() != self._device_index or not ws.is_contiguous():
            raise ValueError(f"the workspace is a contiguous tensor on {self.device}, got one on {ws.device} with strides "
                             f"{ws.stride()}")
        return ws.data_ptr(), ws.nbytes

    def append(self, args: csa_kv_append_args, stream=None) -> None:
        self._call("csa_kv_append", self._append_fn, stream, byref(args))

    def window_attn(self, args: csa_kv_attn_args, ws, stream=None) -> None:
        self._call("csa_window_attn", self._window_fn, stream, byref(args), *self._space(ws))

    def prefix_attn(self, args: csa_kv_attn_args, ws, stream=None) -> None:
        self._call("csa_prefix_attn", self._prefix_fn, stream, byref(args), *self._space(ws))
