"""A paged key-value cache in torch device tensors, for the dense serving path.

``HHRPagedCache`` owns (or is given) the page pools and the workspace, and
forwards to libhhr.so: appending tokens with their rotary positions, and the
attention of one new token per sequence over everything it has.  Which page
belongs to which sequence is the caller's: a table of page indices per
sequence comes with each call.
"""
from __future__ import annotations

import math

import torch

from . import _binding as B
from .rope import check_tensor, on_device

_TYPES = {torch.bfloat16: B.HHR_TYPE_BF16, torch.float16: B.HHR_TYPE_F16, torch.float32: B.HHR_TYPE_F32,
          torch.float8_e4m3fn: B.HHR_TYPE_E4M3}


class HHRPagedCache:
    def __init__(self, *, q_heads, kv_heads, pages=None, page=16, head_dim=128, dtype=torch.bfloat16,
                 kv_dtype=None, layout="head", k_scale=1.0, v_scale=1.0, device="cuda", K=None, V=None):
        """layout: "head" for pools [pages][kv_heads][page][head_dim], "token" for
        [pages][page][kv_heads][head_dim].  dtype (bf16 or fp16): queries and
        appended keys and values; kv_dtype: the pools' (dtype, or
        float8_e4m3fn, whose elements stand for k_scale / v_scale times their
        value).  K, V: pools to use instead of new ones (any strides with adjacent
        elements of a head)."""
        if layout not in ("head", "token"):
            raise ValueError(f'layout must be "head" or "token", got {layout!r}')
        if dtype not in (torch.bfloat16, torch.float16):
            raise ValueError(f"dtype must be bfloat16 or float16, got {dtype}")
        if (K is None) != (V is None):
            raise ValueError("K and V are given together")
        if K is None:
            if pages is None:
                raise ValueError("pages: the size of the pools")
            shape = (pages, kv_heads, page, head_dim) if layout == "head" else (pages, page, kv_heads, head_dim)
            K = torch.zeros(shape, dtype=kv_dtype or dtype, device=device)
            V = torch.zeros_like(K)
        else:
            pages = K.shape[0] if pages is None else pages
            kv_dtype = K.dtype if kv_dtype is None else kv_dtype
            shape = (pages, kv_heads, page, head_dim) if layout == "head" else (pages, page, kv_heads, head_dim)
            check_tensor("K", K, kv_dtype, K.device, shape)
            check_tensor("V", V, kv_dtype, K.device, shape)
            if K.stride(3) != 1 or V.stride(3) != 1:
                raise ValueError("K, V: the elements of a head have to be adjacent")
        if K.dtype not in (dtype, torch.float8_e4m3fn):
            raise ValueError(f"kv_dtype must be {dtype} or float8_e4m3fn, got {K.dtype}")
        self.K, self.V, self.device, self.dtype = K, V, K.device, dtype
        self.scale = 1.0 / math.sqrt(head_dim)
        h, t = (1, 2) if layout == "head" else (2, 1)
        self.desc = B.hhr_paged(q_heads, kv_heads, head_dim, page, pages, 1, 1, _TYPES[dtype], _TYPES[K.dtype],
                                k_scale, v_scale, 0, *(s.stride(i) for s in (K, V) for i in (0, h, t)))
        self._descs = {}
        self.workspace = self.new_workspace()

    def new_workspace(self):
        """A workspace of its own, for attend calls that may run at the same time as others on this cache (another
        stream, another captured graph)."""
        ws = B.hhr_paged_workspace_size(self.desc)
        if ws == 0:
            raise B.HhrError(B.HHR_ERR_INVALID_ARG, "hhr_paged_workspace_size")
        return torch.zeros(ws, dtype=torch.uint8, device=self.device)

    def _table(self, table):
        """The description with this table's columns and row stride, and the table's rows."""
        if table.dim() != 2 or table.dtype != torch.int32 or table.device != self.device or \
                (table.shape[1] > 1 and table.stride(1) != 1):
            raise ValueError(f"table: expected int32 [sequences, pages] on {self.device} with adjacent columns, "
                             f"got {table.dtype} {tuple(table.shape)} on {table.device}")
        rows, cols = table.shape
        stride = table.stride(0) if rows > 1 else cols
        desc = self._descs.get((cols, stride))
        if desc is None:   # never changed after this: another thread's call may be reading it
            desc = B.hhr_paged.from_buffer_copy(self.desc)
            desc.table_cols, desc.table_stride = cols, stride
            if len(self._descs) >= 64:
                self._descs.clear()
            self._descs[cols, stride] = desc
        return desc, rows

    def _rows(self, name, t, heads):
        """Elements between two tokens' rows of t [T, heads, head_dim]."""
        d = self.desc.d
        if t.dim() != 3 or t.shape[1] != heads or t.shape[2] != d or t.dtype != self.dtype or t.device != self.device:
            raise ValueError(f"{name}: expected {self.dtype} [tokens, {heads}, {d}] on {self.device}, "
                             f"got {t.dtype} {tuple(t.shape)} on {t.device}")
        if t.stride(2) != 1 or (heads > 1 and t.stride(1) != d):
            raise ValueError(f"{name}: a token's heads have to be adjacent")
        return t.stride(0)

    def append(self, k, v, positions, table, *, seq=None, q=None, q_out=None, freqs=None, rope_positions=None,
               interleaved=False, mscale=1.0):
        """Stores keys and values [T, kv_heads, head_dim] of T new tokens at places
        positions[t] (int32; negative: a padding row, skipped) of sequences seq[t]
        (rows of `table`; None: token t of sequence t).  freqs (rope_freqs): the keys
        are rotated by rope_positions (None: positions) on the way, and with q
        [T, q_heads, head_dim] the queries too, into q_out (a new tensor if
        None; q itself rotates in place).  Returns q_out."""
        d, rows = self._table(table)
        T = k.shape[0]
        k_row, v_row = self._rows("k", k, d.Hkv), self._rows("v", v, d.Hkv)
        if v.shape[0] != T:
            raise ValueError(f"v: {v.shape[0]} tokens, k has {T}")
        for name, t in (("positions", positions), ("seq", seq), ("rope_positions", rope_positions)):
            if t is None:
                continue
            check_tensor(name, t, torch.int32, self.device, (T,))
            if T > 1 and t.stride(0) != 1:
                raise ValueError(f"{name} has to be contiguous")
        q_tok = o_tok = 0
        if q is not None:
            q_out = torch.empty(q.shape, dtype=q.dtype, device=q.device) if q_out is None else q_out
            q_tok, o_tok = self._rows("q", q, d.Hq), self._rows("q_out", q_out, d.Hq)
            if q.shape[0] != T or q_out.shape[0] != T:
                raise ValueError(f"q, q_out: {q.shape[0]} and {q_out.shape[0]} tokens, k has {T}")
        elif q_out is not None:
            raise ValueError("q_out without q")
        rot = None
        if freqs is not None:
            check_tensor("freqs", freqs, torch.float64, self.device, (freqs.numel(),))
            if not freqs.is_contiguous():
                raise ValueError("freqs has to be contiguous")
            rot = B.hhr_rotation(2 * freqs.numel(), B.HHR_ROPE_INTERLEAVED if interleaved else 0, mscale)
        on_device(self.device, B.hhr_paged_append, d, T, rows, rot, freqs, positions, rope_positions, seq, table,
                  q, q_tok, q_out, o_tok, k, k_row, v, v_row, self.K, self.V, self.workspace)
        return q_out

    def attend(self, q, table, lens, *, out=None, lse=None, window=0, scale=None, workspace=None):
        """Attention of q [B, q_heads, head_dim] over the first lens[b] (int32) tokens of
        each sequence, or the last `window` of them; into out (dtype or float32;
        a new tensor of dtype if None) and lse (float32 [B, q_heads], optional).
        scale: 1/sqrt(head_dim) if None.  workspace (new_workspace): needed by calls that may
        run at the same time as another one on this cache."""
        d, rows = self._table(table)
        q_seq = self._rows("q", q, d.Hq)
        if q.shape[0] != rows:
            raise ValueError(f"q: {q.shape[0]} sequences, table has {rows}")
        check_tensor("lens", lens, torch.int32, self.device, (rows,))
        if rows > 1 and lens.stride(0) != 1:
            raise ValueError("lens has to be contiguous")
        if out is None:
            out = torch.empty(q.shape, dtype=q.dtype, device=q.device)
        elif out.shape != q.shape or out.dtype not in (self.dtype, torch.float32) or out.device != self.device or \
                not out.is_contiguous():
            raise ValueError(f"out: expected a contiguous {self.dtype} or float32 tensor {tuple(q.shape)} on {self.device}")
        if lse is not None:
            check_tensor("lse", lse, torch.float32, self.device, (rows, d.Hq))
            if not lse.is_contiguous():
                raise ValueError("lse has to be contiguous")
        on_device(self.device, B.hhr_paged_attend, d, rows, q, q_seq, self.K, self.V, table, lens, window,
                  self.scale if scale is None else scale, _TYPES[out.dtype], out, lse, self.workspace if workspace is None else workspace, None)
        return out

    def status(self, stream=None, workspace=None) -> int:
        """HHR_OK, or HHR_ERR_BAD_INDEX after a page, sequence or length out of range; cleared after reading."""
        ws = self.workspace if workspace is None else workspace
        if stream is not None:
            return B.hhr_read_status(ws, stream)
        return on_device(self.device, B.hhr_read_status, ws)
