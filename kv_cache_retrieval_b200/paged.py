"""A paged key-value cache in torch device tensors, for the dense serving path.

``HHRPagedCache`` owns (or is given) the page pools and the workspace, and
forwards to libhhr.so: appending tokens with their rotary positions, and the
attention of one new token per sequence over everything it has.  Which page
belongs to which sequence is the caller's: a table of page indices per
sequence comes with each call.
"""
from __future__ import annotations

import ctypes as C
import math
import threading

import torch

from . import _binding as B
from .rope import check_vector, fits, on_device, rotation, written

_TYPES = {torch.bfloat16: B.HHR_TYPE_BF16, torch.float16: B.HHR_TYPE_F16, torch.float32: B.HHR_TYPE_F32,
          torch.float8_e4m3fn: B.HHR_TYPE_E4M3}

_growing = threading.Lock()    # of any cache's workspaces


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
            for name, t in (("K", K), ("V", V)):
                if t.dtype != kv_dtype or t.device != K.device or t.shape != shape:
                    raise ValueError(f"{name}: expected {kv_dtype} {shape} on {K.device}, "
                                     f"got {t.dtype} {tuple(t.shape)} on {t.device}")
            if K.stride(3) != 1 or V.stride(3) != 1:
                raise ValueError("K, V: the elements of a head have to be adjacent")
        if K.dtype not in (dtype, torch.float8_e4m3fn):
            raise ValueError(f"kv_dtype must be {dtype} or float8_e4m3fn, got {K.dtype}")
        self.K, self.V, self.device, self.dtype = K, V, K.device, dtype
        self.scale = 1.0 / math.sqrt(head_dim)
        fits(q_heads, pages)
        h, t = (1, 2) if layout == "head" else (2, 1)
        self.desc = B.hhr_paged(q_heads, kv_heads, head_dim, page, pages, 1, 1, _TYPES[dtype], _TYPES[K.dtype],
                                k_scale, v_scale, 0, *(s.stride(i) for s in (K, V) for i in (0, h, t)))
        self._descs = {}
        self._index, self._Hq, self._Hkv, self._d = K.get_device(), q_heads, kv_heads, head_dim
        self.workspace = self.new_workspace()
        self._spaces = {}

    def _workspace(self):
        """The workspace of the current stream, whose calls follow one another: `workspace` for the first one and for
        captured calls on a stream that had none, one of its own for every other stream."""
        if self._index < 0:
            return self.workspace
        stream = torch._C._cuda_getCurrentRawStream(self._index)
        space = self._spaces.get(stream)
        if space is None:
            with _growing, torch.cuda.device(self._index):
                if torch.cuda.is_current_stream_capturing():    # (a new one would be zeros at the graph's replays only)
                    return self.workspace
                space = self._spaces.setdefault(stream, self.new_workspace() if self._spaces else self.workspace)
        return space

    def new_workspace(self):
        """A workspace of its own, for the attend calls of a captured graph that may run at the same time as others on
        this cache."""
        ws = B.hhr_paged_workspace_size(self.desc)
        if ws == 0:
            raise B.HhrError(B.HHR_ERR_INVALID_ARG, "hhr_paged_workspace_size")
        return torch.zeros(ws, dtype=torch.uint8, device=self.device)

    def _table(self, table):
        """A reference to the description with this table's columns and row stride, and the table's rows."""
        shape, strides = table.shape, table.stride()
        if len(shape) != 2 or table.dtype is not torch.int32 or table.get_device() != self._index or \
                (shape[1] > 1 and strides[1] != 1):
            raise ValueError(f"table: expected int32 [sequences, pages] on {self.device} with adjacent columns, "
                             f"got {table.dtype} {tuple(table.shape)} on {table.device}")
        rows, cols = shape
        stride = strides[0] if rows > 1 else cols
        desc = self._descs.get((cols, stride))
        if desc is None:   # never changed after this: another thread's call may be reading it
            desc = B.hhr_paged.from_buffer_copy(self.desc)
            desc.table_cols, desc.table_stride = fits(cols, stride)
            if len(self._descs) >= 64:
                self._descs.clear()
            desc = self._descs[cols, stride] = C.byref(desc)
        return desc, rows

    def _rows(self, name, t, heads):
        """T of t [T, heads, head_dim] and the elements between two of its rows."""
        d, shape = self._d, t.shape
        if len(shape) != 3 or t.dtype is not self.dtype or t.get_device() != self._index or shape[1] != heads or shape[2] != d:
            raise ValueError(f"{name}: expected {self.dtype} [tokens, {heads}, {d}] on {self.device}, "
                             f"got {t.dtype} {tuple(t.shape)} on {t.device}")
        row, head, one = t.stride()
        if one != 1 or (heads > 1 and head != d):
            raise ValueError(f"{name}: a token's heads have to be adjacent")
        if shape[0] >> 31:
            fits(shape[0])
        return shape[0], row

    def append(self, k, v, positions, table, *, seq=None, q=None, q_out=None, freqs=None, rope_positions=None,
               interleaved=False, mscale=1.0):
        """Stores keys and values [T, kv_heads, head_dim] of T new tokens at places
        positions[t] (int32; negative: a padding row, skipped) of sequences seq[t]
        (rows of `table`; None: token t of sequence t).  freqs (rope_freqs): the keys
        are rotated by rope_positions (None: positions) on the way, and with q
        [T, q_heads, head_dim] the queries too, into q_out (a new tensor if
        None, whose skipped rows hold nothing in particular; q itself rotates in place).  Returns q_out.  Writes the pools in place: no
        gradient passes through it."""
        index = self._index
        desc, rows = self._table(table)
        T, k_row = self._rows("k", k, self._Hkv)
        v_T, v_row = self._rows("v", v, self._Hkv)
        if v_T != T:
            raise ValueError(f"v: {v_T} tokens, k has {T}")
        check_vector("positions", positions, torch.int32, T, index)
        if seq is not None:
            check_vector("seq", seq, torch.int32, T, index)
        if rope_positions is not None:
            check_vector("rope_positions", rope_positions, torch.int32, T, index)
        q_tok = o_tok = 0
        if q is not None:
            if q_out is None:
                q_out = q.new_empty(q.shape)
            q_T, q_tok = self._rows("q", q, self._Hq)
            o_T, o_tok = self._rows("q_out", q_out, self._Hq)
            if q_T != T or o_T != T:
                raise ValueError(f"q, q_out: {q_T} and {o_T} tokens, k has {T}")
        elif q_out is not None:
            raise ValueError("q_out without q")
        rot = None
        if freqs is not None:
            half = freqs.numel()
            check_vector("freqs", freqs, torch.float64, half, index)
            rot = rotation(2 * half, B.HHR_ROPE_INTERLEAVED if interleaved else 0, mscale)
        written((self.K, self.V) if q is None else (self.K, self.V, q_out))
        st = on_device(index, B.lib().hhr_paged_append, desc, T, rows, rot, None if freqs is None else freqs.data_ptr(),
                       positions.data_ptr(), None if rope_positions is None else rope_positions.data_ptr(),
                       None if seq is None else seq.data_ptr(), table.data_ptr(), None if q is None else q.data_ptr(), q_tok,
                       None if q is None else q_out.data_ptr(), o_tok, k.data_ptr(), k_row, v.data_ptr(), v_row,
                       self.K.data_ptr(), self.V.data_ptr(), self.workspace.data_ptr())
        if st:
            raise B.HhrError(st, "hhr_paged_append")
        return q_out

    def attend(self, q, table, lens, *, out=None, lse=None, window=0, scale=None, workspace=None):
        """Attention of q [B, q_heads, head_dim] over the first lens[b] (int32) tokens of
        each sequence, or the last `window` of them; into out (dtype or float32;
        a new tensor of dtype if None) and lse (float32 [B, q_heads], optional).
        scale: 1/sqrt(head_dim) if None.  workspace (new_workspace): needed by a captured call that may run
        at the same time as another call on this cache; calls on several streams have one each.  lens and table
        must not change while the call runs (hhr.h, hhr_paged_attend).  A serving call: it has no gradient."""
        index = self._index
        desc, rows = self._table(table)
        q_B, q_seq = self._rows("q", q, self._Hq)
        if q_B != rows:
            raise ValueError(f"q: {q_B} sequences, table has {rows}")
        check_vector("lens", lens, torch.int32, rows, index)
        if out is None:
            out = q.new_empty(q.shape)
        elif out.shape != q.shape or (out.dtype is not self.dtype and out.dtype is not torch.float32) or \
                out.get_device() != index or not out.is_contiguous():
            raise ValueError(f"out: expected a contiguous {self.dtype} or float32 tensor {tuple(q.shape)} on {self.device}")
        if lse is not None and (lse.dtype is not torch.float32 or lse.shape != (rows, self._Hq) or
                                lse.get_device() != index or not lse.is_contiguous()):
            raise ValueError(f"lse: expected a contiguous float32 tensor [{rows}, {self._Hq}] on {self.device}")
        if window >> 31:      # no sequence is that long
            window = (1 << 31) - 1 if window > 0 else -1
        if workspace is None:
            workspace = self._workspace()
        elif workspace.get_device() != index or not workspace.is_contiguous():
            raise ValueError(f"workspace: expected a contiguous tensor on {self.device}")
        written((out,) if lse is None else (out, lse))
        st = on_device(index, B.lib().hhr_paged_attend, desc, rows, q.data_ptr(), q_seq, self.K.data_ptr(), self.V.data_ptr(),
                       table.data_ptr(), lens.data_ptr(), window, self.scale if scale is None else scale, _TYPES[out.dtype],
                       out.data_ptr(), None if lse is None else lse.data_ptr(), workspace.data_ptr(),
                       workspace.numel() * workspace.element_size())
        if st:
            raise B.HhrError(st, "hhr_paged_attend")
        return out

    def status(self, stream=None, workspace=None) -> int:
        """HHR_OK, or HHR_ERR_BAD_INDEX after a page, sequence or length out of range; cleared after reading.  Waits for
        `stream` (the current one if None); without a workspace, that of every stream is read."""
        with torch.cuda.device(self.device):
            if workspace is not None:
                return B.hhr_read_status(workspace, stream)
            with _growing:
                spaces = {id(w): w for w in (self.workspace, *self._spaces.values())}.values()
            return max(B.hhr_read_status(w, stream) for w in spaces)
