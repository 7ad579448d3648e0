"""Torch-facing helpers over the C ABI: a paged KV cache that owns its device
tensors, and the host page allocator.

PyTorch only allocates device memory and supplies the stream; every step of
append, scoring, selection and attention runs in libpkv's kernels.
"""
from __future__ import annotations

import contextlib
import ctypes
import math
import threading
from typing import Dict, Optional, Tuple

import numpy as np
import torch

from . import binding as B

_TORCH_TO_PKV = {torch.float16: B.F16, torch.bfloat16: B.BF16, torch.float32: B.F32}
_NAME_TO_PKV = {"f16": B.F16, "bf16": B.BF16, "int8": B.I8, "u4": B.U4}
_PKV_TO_TORCH = {B.F16: torch.float16, B.BF16: torch.bfloat16, B.F32: torch.float32, B.I8: torch.uint8,
                 B.U4: torch.uint8}   # I8 pools hold the bytes u = code + 128
_QUANT = {"none": B.QUANT_NONE, "per_token": B.QUANT_PER_TOKEN, "per_group64": B.QUANT_PER_GROUP64}


def pkv_dtype(t: torch.Tensor) -> int:
    try:
        return _TORCH_TO_PKV[t.dtype]
    except KeyError:
        raise TypeError(f"unsupported dtype {t.dtype}") from None


def _ptr(t: Optional[torch.Tensor]) -> int:
    return 0 if t is None else t.data_ptr()


def _stream(stream: Optional[torch.cuda.Stream]) -> int:
    s = stream if stream is not None else torch.cuda.current_stream()
    return s.cuda_stream


def _need(t: torch.Tensor, name: str, dtype=None, device=None) -> None:
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if device is not None and t.device != device:
        raise ValueError(f"{name} must be on {device}")


def _host_ids(ids, name: str) -> np.ndarray:
    """Page or row ids on the host as contiguous int32 (a list, an array or a CPU tensor)."""
    if type(ids) is np.ndarray and ids.dtype == np.int32 and ids.ndim == 1 and ids.flags.c_contiguous:
        return ids
    if isinstance(ids, torch.Tensor):
        if ids.is_cuda:
            raise ValueError(f"{name} must be on the host")
        ids = ids.numpy()
    a = np.asarray(ids)
    if a.size == 0:
        a = a.astype(np.int32)
    if a.ndim != 1 or a.dtype.kind not in "iu":
        raise TypeError(f"{name} must be a list of whole numbers")
    if a.dtype != np.int32:
        if a.size and (int(a.min()) < 0 or int(a.max()) > 0x7FFFFFFF):
            raise ValueError(f"{name} holds an id out of range")
        a = a.astype(np.int32)
    return np.ascontiguousarray(a)


def _pair_ids(src, dst, what: str) -> Tuple[np.ndarray, np.ndarray]:
    s, d = _host_ids(src, f"src_{what}"), _host_ids(dst, f"dst_{what}")
    if s.size != d.size:
        raise ValueError(f"{s.size} source and {d.size} destination {what}")
    return s, d


def _addr(a: np.ndarray) -> int:
    return a.__array_interface__["data"][0]


# torch's own way to the current stream's handle; the public one makes a Stream object
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or \
    (lambda index: torch.cuda.current_stream(index).cuda_stream)
_capturing = getattr(torch._C, "_cuda_isCurrentStreamCapturing", None) or torch.cuda.is_current_stream_capturing
_same_device = contextlib.nullcontext()


class PagedKVCache:
    """One layer's paged K/V pools (see pkv_cache in include/pkv.h for layouts)."""

    def __init__(self, num_pages: int, page_size: int, num_kv_heads: int, head_dim: int,
                 kv_dtype: str = "bf16", quant: str = "none", with_meta: bool = False,
                 tail_rows: int = 0, device: str = "cuda", poison: bool = False):
        self.num_pages, self.page_size = num_pages, page_size
        self.num_kv_heads, self.head_dim = num_kv_heads, head_dim
        self.kv_dtype, self.quant = _NAME_TO_PKV[kv_dtype], _QUANT[quant]
        self.device = torch.device(device)
        tdt = _PKV_TO_TORCH[self.kv_dtype]
        # 4-bit codes: two per byte
        shape = (num_pages, num_kv_heads, page_size, head_dim // 2 if self.kv_dtype == B.U4 else head_dim)
        self.k_pages = torch.empty(shape, dtype=tdt, device=self.device)
        self.v_pages = torch.empty(shape, dtype=tdt, device=self.device)
        self.device = self.k_pages.device      # concrete index (cuda:N)
        self.kv_sz = None
        self.tail = None
        if self.kv_dtype in (B.I8, B.U4):
            gran = 1 if self.quant == B.QUANT_PER_TOKEN else 64
            self.kv_sz = torch.empty((num_pages, num_kv_heads, page_size // gran, 4),
                                     dtype=torch.float32, device=self.device)
            if self.quant == B.QUANT_PER_GROUP64:
                rows = max(1, tail_rows)
                self.tail = torch.zeros((rows, num_kv_heads, 2, 2, 64, head_dim),
                                        dtype=torch.float32, device=self.device)
        self.page_meta = (torch.empty((num_pages, num_kv_heads, 2, head_dim), dtype=torch.float32,
                                      device=self.device) if with_meta else None)
        if poison:
            # unwritten slots read as NaN (float) / NaN scales (INT8): a stray read shows
            if self.kv_dtype in (B.I8, B.U4):
                self.k_pages.fill_(0)
                self.v_pages.fill_(0)
                self.kv_sz.fill_(float("nan"))
            else:
                self.k_pages.fill_(float("nan"))
                self.v_pages.fill_(float("nan"))
            if self.page_meta is not None:
                self.page_meta.fill_(float("nan"))
        self._describe()

    def _describe(self) -> None:
        self._desc = B.PkvCache(
            self.num_pages, self.page_size, self.num_kv_heads, self.head_dim, self.kv_dtype, self.quant,
            self.k_pages.data_ptr(), self.v_pages.data_ptr(), _ptr(self.kv_sz), _ptr(self.tail),
            0 if self.tail is None else self.tail.shape[0], _ptr(self.page_meta))
        self._ws: Dict[Tuple, torch.Tensor] = {}
        self._shared_ws: Dict[int, torch.Tensor] = {}     # by stream
        self._shared_fit: Dict[Tuple[int, int, int, int], torch.Tensor] = {}   # the same, by stream and shape
        self._shared_lent: Dict[int, torch.Tensor] = {}   # by address
        self._shared_lock = threading.Lock()

    @classmethod
    def from_pools(cls, k_pages: torch.Tensor, v_pages: torch.Tensor, kv_dtype: str = "bf16",
                   quant: str = "none", kv_sz: Optional[torch.Tensor] = None,
                   tail: Optional[torch.Tensor] = None,
                   page_meta: Optional[torch.Tensor] = None) -> "PagedKVCache":
        """A cache over pools that the caller has (layouts as in include/pkv.h); they are
        kept alive, not copied."""
        self = cls.__new__(cls)
        self.kv_dtype, self.quant = _NAME_TO_PKV[kv_dtype], _QUANT[quant]
        if k_pages.dim() != 4:
            raise ValueError("k_pages must be [pages][kv heads][page size][row]")
        self.num_pages, self.num_kv_heads, self.page_size, row = k_pages.shape
        self.head_dim = 2 * row if self.kv_dtype == B.U4 else row
        self.device = k_pages.device
        N, H, ps, d = self.num_pages, self.num_kv_heads, self.page_size, self.head_dim
        gran = 0 if quant == "none" else (1 if quant == "per_token" else 64)
        want = [("k_pages", k_pages, _PKV_TO_TORCH[self.kv_dtype], (N, H, ps, row)),
                ("v_pages", v_pages, _PKV_TO_TORCH[self.kv_dtype], (N, H, ps, row)),
                ("kv_sz", kv_sz, torch.float32, (N, H, ps // gran, 4) if gran else None),
                ("tail", tail, torch.float32, (-1, H, 2, 2, 64, d) if gran == 64 else None),
                ("page_meta", page_meta, torch.float32, (N, H, 2, d))]
        for name, t, dtype, shape in want:
            if t is None:
                if name == "kv_sz" and gran:
                    raise ValueError(f"{quant} caches need kv_sz")
                continue
            if shape is None:
                raise ValueError(f"a cache with quant={quant!r} has no {name}")
            _need(t, name, dtype, self.device)
            if t.dim() != len(shape) or any(s not in (-1, n) for s, n in zip(shape, t.shape)):
                raise ValueError(f"{name} must be {list(shape)}, got {list(t.shape)}")
        self.k_pages, self.v_pages, self.kv_sz, self.tail, self.page_meta = k_pages, v_pages, kv_sz, tail, page_meta
        self._describe()
        return self

    def descriptor(self) -> B.PkvCache:
        return self._desc

    # ------------------------------------------------------------------ append
    def append(self, k_new: torch.Tensor, v_new: torch.Tensor, block_table: torch.Tensor,
               positions: torch.Tensor, new_lens: Optional[torch.Tensor] = None,
               dev_status: Optional[torch.Tensor] = None,
               stream: Optional[torch.cuda.Stream] = None) -> None:
        """Write tokens k_new/v_new [B][T][Hkv][d] at positions[b] .. (+new_lens[b])."""
        for t, n in ((k_new, "k_new"), (v_new, "v_new")):
            _need(t, n, device=self.device)
        _need(block_table, "block_table", torch.int32, self.device)
        _need(positions, "positions", torch.int32, self.device)
        if new_lens is not None:
            _need(new_lens, "new_lens", torch.int32, self.device)
        Bsz, T = k_new.shape[0], k_new.shape[1]
        B.kv_append(self._desc, Bsz, T, k_new.data_ptr(), v_new.data_ptr(), pkv_dtype(k_new),
                    block_table.data_ptr(), block_table.shape[1], positions.data_ptr(),
                    _ptr(new_lens), _ptr(dev_status), _stream(stream))

    # ----------------------------------------------------------- score / top-K
    def score_topk(self, q: torch.Tensor, block_table: torch.Tensor, seq_lens: torch.Tensor,
                   top_k: int, want_scores: bool = False, dev_status: Optional[torch.Tensor] = None,
                   sel: Optional[torch.Tensor] = None, count: Optional[torch.Tensor] = None,
                   scores: Optional[torch.Tensor] = None,
                   stream: Optional[torch.cuda.Stream] = None, group_mode: int = 0,
                   early_start: bool = False):
        """Top-K pages per row: per (sequence, query head), or with group_mode 1 / 2
        (sum / max of the group's scores) per (sequence, kv head). Returns
        (sel [B][R][K], count [B][R], scores [B][R][max_pages] or None).

        early_start: the kernel launched just before on the stream writes nothing
        this call reads (q, tables, lengths, boxes), so the scoring starts under it."""
        _need(q, "q", device=self.device)
        Bsz, Hq = q.shape[0], q.shape[1]
        R = Hq if group_mode == 0 else self.num_kv_heads
        mp = block_table.shape[1]
        if sel is None:
            sel = torch.empty((Bsz, R, top_k), dtype=torch.int32, device=self.device)
        if count is None:
            count = torch.empty((Bsz, R), dtype=torch.int32, device=self.device)
        if want_scores and scores is None:
            scores = torch.empty((Bsz, R, mp), dtype=torch.float32, device=self.device)
        B.page_score_topk(self._desc, Bsz, Hq, q.data_ptr(), pkv_dtype(q), block_table.data_ptr(),
                          mp, seq_lens.data_ptr(), top_k, sel.data_ptr(), count.data_ptr(),
                          _ptr(scores), _ptr(dev_status), _stream(stream), group_mode=group_mode,
                          early_start=1 if early_start else 0)
        return sel, count, scores

    # --------------------------------------------------------------- attention
    def workspace(self, batch: int, num_q_heads: int, sparse: int, num_splits: int) -> torch.Tensor:
        """Zero-filled workspace of at least the size the library asks for (kept and reused).
        sparse: 0 dense, 1 page lists per query head, 2 lists shared by each group."""
        key = (batch, num_q_heads, int(sparse), num_splits)
        n = B.attention_workspace_bytes(self._desc, batch, num_q_heads, sparse, num_splits)
        ws = self._ws.get(key)
        if ws is None or ws.numel() < n:
            ws = torch.zeros(n, dtype=torch.uint8, device=self.device)
            self._ws[key] = ws
        return ws

    def attention(self, q: torch.Tensor, block_table: torch.Tensor, seq_lens: torch.Tensor,
                  sm_scale: Optional[float] = None, sel: Optional[torch.Tensor] = None,
                  sel_count: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None,
                  out_dtype: torch.dtype = torch.float32, num_splits: int = 0,
                  dev_status: Optional[torch.Tensor] = None,
                  stream: Optional[torch.cuda.Stream] = None, fresh_rows: int = -1,
                  sel_shared: bool = False) -> torch.Tensor:
        """Decode attention for q [B][Hq][d]; dense, or over sel[b][h][:sel_count[b][h]] pages.

        fresh_rows >= 0 lets the call start while the kernel launched just before
        it on the stream still runs, on the promise that, of this call's inputs,
        that kernel writes only the K/V rows of the last fresh_rows tokens of each
        sequence (e.g. the kv_append of this step, fresh_rows = its token count;
        0 after another attention call)."""
        _need(q, "q", device=self.device)
        _need(block_table, "block_table", torch.int32, self.device)
        _need(seq_lens, "seq_lens", torch.int32, self.device)
        Bsz, Hq, d = q.shape
        if sm_scale is None:
            sm_scale = 1.0 / float(np.sqrt(d))
        if out is None:
            out = torch.empty((Bsz, Hq, d), dtype=out_dtype, device=self.device)
        sparse = sel is not None
        mode = 0 if not sparse else (2 if sel_shared else 1)
        ws = self.workspace(Bsz, Hq, mode, num_splits)
        B.paged_decode_attention(
            self._desc, Bsz, Hq, q.data_ptr(), pkv_dtype(q), float(sm_scale),
            block_table.data_ptr(), block_table.shape[1], seq_lens.data_ptr(), _ptr(sel),
            _ptr(sel_count), sel.shape[2] if sparse else 0, out.data_ptr(), pkv_dtype(out),
            num_splits, ws.data_ptr(), ws.numel(), _ptr(dev_status), _stream(stream),
            fresh_rows=fresh_rows, sel_shared=1 if (sparse and sel_shared) else 0)
        return out

    def append_attention(self, k_new: torch.Tensor, v_new: torch.Tensor, q: torch.Tensor,
                         block_table: torch.Tensor, seq_lens: torch.Tensor, sm_scale: Optional[float] = None,
                         out: Optional[torch.Tensor] = None, out_dtype: torch.dtype = torch.float32,
                         num_splits: int = 0, dev_status: Optional[torch.Tensor] = None,
                         stream: Optional[torch.cuda.Stream] = None, fresh_rows: int = -1) -> torch.Tensor:
        """One decode step: write k_new / v_new [B][Hkv][d] (each sequence's token at
        position seq_lens[b] - 1) and attend over [0, seq_lens[b]), in one call."""
        _need(q, "q", device=self.device)
        _need(k_new, "k_new", device=self.device)
        _need(v_new, "v_new", device=self.device)
        _need(block_table, "block_table", torch.int32, self.device)
        _need(seq_lens, "seq_lens", torch.int32, self.device)
        Bsz, Hq, d = q.shape
        if sm_scale is None:
            sm_scale = 1.0 / float(np.sqrt(d))
        if out is None:
            out = torch.empty((Bsz, Hq, d), dtype=out_dtype, device=self.device)
        ws = self.workspace(Bsz, Hq, 0, num_splits)
        src = B.BF16 if k_new.dtype == torch.bfloat16 else B.F16
        B.append_decode_attention(
            self._desc, Bsz, Hq, k_new.data_ptr(), v_new.data_ptr(), src, q.data_ptr(), pkv_dtype(q),
            float(sm_scale), block_table.data_ptr(), block_table.shape[1], seq_lens.data_ptr(),
            out.data_ptr(), pkv_dtype(out), num_splits, fresh_rows, ws.data_ptr(), ws.numel(),
            _ptr(dev_status), _stream(stream))
        return out


    # --------------------------------------------------- sequences that share pages
    # (these calls may take less time on the device than their checks here: they are written
    # for few Python operations)
    def _on_device(self):
        """Context in which the cache's device is the current one."""
        if torch.cuda.current_device() == self.device.index:
            return _same_device
        return torch.cuda.device(self.device)

    def _launch_stream(self, stream: Optional[torch.cuda.Stream]) -> int:
        return _raw_stream(self.device.index) if stream is None else stream.cuda_stream

    def copy_pages(self, src_pages, dst_pages, src_rows=None, dst_rows=None,
                   stream: Optional[torch.cuda.Stream] = None) -> None:
        """Page dst_pages[i] becomes a copy of page src_pages[i] (K, V, scales, boxes), and
        tail row dst_rows[i] of row src_rows[i] (per-group caches). The ids are on the host:
        lists, int32 arrays or CPU tensors, as PageAllocator.unshare and .compact give them."""
        sp, dp = _pair_ids(src_pages, dst_pages, "pages")
        if src_rows is None and dst_rows is None:
            n_rows = sr = dr = 0
        else:
            rows = _pair_ids(() if src_rows is None else src_rows, () if dst_rows is None else dst_rows, "rows")
            n_rows, sr, dr = rows[0].size, _addr(rows[0]), _addr(rows[1])
        with self._on_device():
            B.copy_pages(self._desc, sp.size, _addr(sp), _addr(dp), n_rows, sr, dr, self._launch_stream(stream))

    def remap_table(self, block_table: torch.Tensor, src_pages, dst_pages,
                    stream: Optional[torch.cuda.Stream] = None) -> None:
        """Entries of block_table equal to src_pages[i] become dst_pages[i] (in place)."""
        _need(block_table, "block_table", torch.int32, self.device)
        if block_table.dim() != 2:
            raise ValueError("block_table must be [batch][pages]")
        sp, dp = _pair_ids(src_pages, dst_pages, "pages")
        if block_table.numel() == 0:
            return
        with self._on_device():
            B.remap_block_table(block_table.data_ptr(), block_table.shape[0], block_table.shape[1],
                                self.num_pages, sp.size, _addr(sp), _addr(dp), self._launch_stream(stream))

    def shared_workspace(self, batch: int, num_q_heads: int, num_splits: int = 0,
                         stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
        """A workspace large enough for shared_attention with these shapes: the stream's own, which
        the cache also uses by default, until a larger call needs a larger one. It is kept alive
        as long as the cache (a captured graph may refer to it). During a capture: memory of the
        graph's pool."""
        with self._on_device() if stream is None else torch.cuda.stream(stream):
            ws = self._shared_workspace(batch, num_q_heads, num_splits, _raw_stream(self.device.index))
            if not _capturing():
                self._shared_lent[ws.data_ptr()] = ws
        return ws

    def _shared_workspace(self, batch: int, num_q_heads: int, num_splits: int, stream: int) -> torch.Tensor:
        capturing = _capturing()
        key = (stream, batch, num_q_heads, num_splits)
        ws = self._shared_fit.get(key)
        if ws is not None and not capturing:
            return ws
        n = B.shared_prefix_workspace_bytes(self._desc, batch, num_q_heads, num_splits)
        if capturing:
            # from the graph's memory pool and this call's alone: graphs share it with nothing that
            # could run beside them, and it goes when they go
            return torch.empty(n, dtype=torch.uint8, device=self.device)
        # One per stream, of any contents. A quarter more at a time, so that those lent out and
        # outgrown add up to a few times the largest at most.
        ws = self._shared_ws.get(stream)
        if ws is None or ws.numel() < n:
            if ws is not None:
                n = max(n, ws.numel() + ws.numel() // 4)
            ws = self._shared_ws[stream] = torch.empty(n, dtype=torch.uint8, device=self.device)
            self._shared_fit.clear()
        self._shared_fit[key] = ws
        return ws

    def shared_attention(self, q: torch.Tensor, block_table: torch.Tensor, seq_lens: torch.Tensor,
                         prefix_group: torch.Tensor, prefix_lens: torch.Tensor,
                         sm_scale: Optional[float] = None, out: Optional[torch.Tensor] = None,
                         out_dtype: torch.dtype = torch.float32, num_splits: int = 0,
                         dev_status: Optional[torch.Tensor] = None,
                         stream: Optional[torch.cuda.Stream] = None,
                         workspace: Optional[torch.Tensor] = None) -> torch.Tensor:
        """Decode attention for q [B][Hq][d] where the rows of group g (prefix_group [B], -1:
        none) have their first prefix_lens[g] tokens in common, which are then read once.
        Results are those of attention() up to rounding: with a 16-bit out_dtype softmax weights
        may be rounded once to q's type, where attention() keeps more; see
        pkv_shared_prefix_attention in include/pkv.h. q is f16 or bf16, for 16-bit caches of the
        cache's type.

        workspace: memory of shared_workspace()'s size for this call alone. By default the calls
        of a stream share one that grows with them, and a call that torch.cuda.graph captures
        has its own in the graph's memory pool. (A capture that does not go through
        torch.cuda.graph needs the argument: nothing would keep the call's own memory.) Threads
        that call on the same stream with an argument of their own each need separate ones.
        stream: the call's, and that of the memory it allocates; the current one by default."""
        if stream is not None:
            # (memory allocated on another stream may still be in use there)
            with torch.cuda.stream(stream):
                return self.shared_attention(q, block_table, seq_lens, prefix_group, prefix_lens, sm_scale, out,
                                             out_dtype, num_splits, dev_status, None, workspace)
        index = -1 if self.device.index is None else self.device.index
        for t, n in ((q, "q"), (block_table, "block_table"), (seq_lens, "seq_lens"), (prefix_group, "prefix_group"),
                     (prefix_lens, "prefix_lens")):
            if t.get_device() != index or not t.is_contiguous() or (t is not q and t.dtype is not torch.int32):
                _need(t, n, None if t is q else torch.int32, self.device)
        if q.dim() != 3 or block_table.dim() != 2 or prefix_lens.dim() != 1:
            raise ValueError("q must be [batch][heads][channels], block_table [batch][pages], prefix_lens [groups]")
        Bsz, Hq, d = q.shape
        rows, width = block_table.shape
        if d != self.head_dim or rows != Bsz or seq_lens.shape != (Bsz,) or prefix_group.shape != (Bsz,):
            raise ValueError(f"for q {list(q.shape)} and head_dim {self.head_dim}: block_table {list(block_table.shape)}, "
                             f"seq_lens {list(seq_lens.shape)}, prefix_group {list(prefix_group.shape)}")
        if out is None:
            out = torch.empty((Bsz, Hq, d), dtype=out_dtype, device=self.device)
        else:
            _need(out, "out", None, self.device)
            if out.shape != q.shape:
                raise ValueError(f"out must be {list(q.shape)}, got {list(out.shape)}")
        with self._on_device():
            st = _raw_stream(self.device.index)
            if workspace is None:
                ws = self._shared_workspace(Bsz, Hq, num_splits, st)
            else:
                ws = workspace
                _need(ws, "workspace", None, self.device)
            with self._shared_lock:   # a call's two launches follow one another on the stream
                B.shared_prefix_attention(
                    self._desc, Bsz, Hq, q.data_ptr(), pkv_dtype(q),
                    1.0 / math.sqrt(d) if sm_scale is None else float(sm_scale), block_table.data_ptr(), width,
                    seq_lens.data_ptr(), prefix_group.data_ptr(), prefix_lens.data_ptr(), prefix_lens.shape[0],
                    out.data_ptr(), pkv_dtype(out), num_splits, ws.data_ptr(), ws.nbytes, _ptr(dev_status), st)
        return out


class PageAllocator:
    """Host free-list page allocator of libpkv (pkv_alloc_*)."""

    def __init__(self, num_pages: int):
        self._h = B.alloc_create(num_pages)
        self.num_pages = num_pages

    def reserve(self, seq_id: int, total_tokens: int, page_size: int, max_pages: int) -> np.ndarray:
        row = np.full(max_pages, -1, dtype=np.int32)
        B.alloc_reserve(self._h, seq_id, total_tokens, page_size,
                        row.ctypes.data_as(ctypes.c_void_p).value, max_pages)
        return row

    def free(self, seq_id: int) -> None:
        B.alloc_free(self._h, seq_id)

    def fork(self, parent: int, child: int, tokens: int, page_size: int, max_pages: int) -> np.ndarray:
        """Sequence child shares the pages of parent's first `tokens` tokens; its table row."""
        row = np.full(max_pages, -1, dtype=np.int32)
        B.alloc_fork(self._h, parent, child, tokens, page_size, row.ctypes.data, max_pages)
        return row

    def unshare(self, seq_id: int, first_token: int, page_size: int,
                max_pages: int) -> Tuple[np.ndarray, np.ndarray, np.ndarray]:
        """Pages of its own for seq_id from first_token's page on: (source pages, destination
        pages) for PagedKVCache.copy_pages, and the sequence's new table row."""
        row = np.full(max_pages, -1, dtype=np.int32)
        src, dst = np.empty(max_pages, dtype=np.int32), np.empty(max_pages, dtype=np.int32)
        n = B.alloc_unshare(self._h, seq_id, first_token, page_size, max_pages, src.ctypes.data,
                            dst.ctypes.data, row.ctypes.data, max_pages)
        return src[:n], dst[:n], row

    def compact(self, max_moves: Optional[int] = None) -> Tuple[np.ndarray, np.ndarray]:
        """Move the pages in use to the lowest ids: (source pages, destination pages) for
        PagedKVCache.copy_pages and .remap_table."""
        m = self.num_pages if max_moves is None else max_moves
        size = max(0, min(m, self.num_pages))
        src, dst = np.empty(size, dtype=np.int32), np.empty(size, dtype=np.int32)
        n = B.alloc_compact(self._h, m if m < 0 else size, src.ctypes.data, dst.ctypes.data)
        return src[:n], dst[:n]

    def table(self, seq_id: int, max_pages: int) -> np.ndarray:
        row = np.full(max_pages, -1, dtype=np.int32)
        B.alloc_table(self._h, seq_id, row.ctypes.data, max_pages)
        return row

    def page_refs(self, page: int) -> int:
        """Sequences that own a page."""
        return B.alloc_page_refs(self._h, page)

    @property
    def num_free(self) -> int:
        return B.alloc_num_free(self._h)

    def seq_pages(self, seq_id: int) -> int:
        return B.alloc_seq_pages(self._h, seq_id)

    def check(self) -> int:
        return B.alloc_check(self._h)

    def close(self) -> None:
        if self._h:
            B.alloc_destroy(self._h)
            self._h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass
