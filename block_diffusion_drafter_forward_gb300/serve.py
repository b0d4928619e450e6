"""Serving operators around the drafter, over torch device tensors: page tables and row maps built
on the device (`extend_tables`), K/V rows appended to a paged cache and attended over (`PagedKV`),
and tokens drawn from logits (`sample`).  Thin calls of dflash_extend_tables, dflash_append_kv,
dflash_attend and dflash_sample: include/dflash.h states what each computes and refuses.

Every call is asynchronous on `stream` (default: the current stream of the tensors' device), copies
nothing to the host and keeps nothing for the next call.  Outputs and workspaces that a call
allocates itself belong to that stream.  The kernels report bad page ids, lengths and full pools in
one status word per device, read and cleared by `serve_status`.  Nothing here records gradients."""
from __future__ import annotations

import ctypes
import math
import threading
from typing import Dict, NamedTuple, Optional, Tuple

import torch

from . import _lib as L

_I32, _F32, _BF16 = torch.int32, torch.float32, torch.bfloat16
_INT_MAX = 2 ** 31 - 1  # larger numbers would be cut to 32 bits on the way into the library
_status: Dict[int, torch.Tensor] = {}  # device index -> its status word
_status_lock = threading.Lock()


class RowPlan(NamedTuple):
    """What `extend_tables` returns: rows of a step and where they go (int32 device tensors)."""
    kv_lens: torch.Tensor     # [nb] rows of each sequence, the new ones included
    row_starts: torch.Tensor  # [nb + 1] first new row of each sequence in the step; the last: total
    row_seq: torch.Tensor     # [max_rows] sequence of each new row, -1 past the total
    row_index: torch.Tensor   # [max_rows] its row (and position) in the sequence, -1 past the total
    slots: torch.Tensor       # [max_rows] its slot in the cache, -1 past the total
    free_end: torch.Tensor    # [1] position in the stack of free pages after this step


def _status_word(device: torch.device) -> torch.Tensor:
    w = _status.get(device.index)
    if w is None:
        with _status_lock:
            w = _status.get(device.index)
            if w is None:
                if torch.cuda.is_current_stream_capturing():
                    raise RuntimeError("the first serving call of a device (or serve_status()) must come before a capture")
                with torch.inference_mode(False):  # it outlives the caller's mode
                    w = torch.zeros(1, dtype=_I32, device=device)
                torch.cuda.current_stream(device).synchronize()  # zeroed for every stream
                _status[device.index] = w
    return w


def serve_status(device=None, stream: Optional[torch.cuda.Stream] = None) -> int:
    """Synchronise `stream` (default: the current one), read the device's DFLASH_DEV_* bits of the
    serving calls since the last read, and clear them: at once, so that a call on another stream
    meanwhile loses none of its own."""
    device = torch.device("cuda", torch.cuda.current_device()) if device is None else torch.device(device)
    if device.index is None:
        device = torch.device("cuda", torch.cuda.current_device())
    with _on(device, stream) as st:
        flags = torch.empty(1, dtype=_I32, device=device)
        L.dflash_take_status(_status_word(device).data_ptr(), flags.data_ptr(), st)
        return int(flags.item())


def _first(t, name: str, dim: int, dtypes=(_I32,)) -> torch.Tensor:
    """The tensor whose device and sizes the others of a call are held to."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name}: expected a torch.Tensor, got {type(t).__name__}")
    if t.device.type != "cuda":
        raise ValueError(f"{name}: expected a cuda tensor, got one on {t.device}")
    if t.dtype not in dtypes:
        raise ValueError(f"{name}: expected {' or '.join(map(str, dtypes))}, got {t.dtype}")
    if t.dim() != dim:
        raise ValueError(f"{name}: expected {dim} dimensions, got {t.dim()}")
    return t


def _refuse(t, name: str, dtype: torch.dtype, shape: Tuple[int, ...], device: torch.device) -> None:
    """Raises for what keeps `t` from being a `dtype` tensor of `shape` on `device` with its rows contiguous."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name}: expected a torch.Tensor, got {type(t).__name__}")
    if t.device != device:
        raise ValueError(f"{name}: expected a tensor on {device}, got one on {t.device}")
    if t.dtype is not dtype:
        raise ValueError(f"{name}: expected {dtype}, got {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name}: expected shape {tuple(shape)}, got {tuple(t.shape)}")
    raise ValueError(f"{name}: must be contiguous")


def _i32(n: int, name: str) -> int:
    if n > _INT_MAX:
        raise ValueError(f"{name}: {n} are too many for one call")
    return n


def _limit(n) -> int:
    """A limit for the library: beyond 32 bits as good as the largest, below zero refused there."""
    return max(-1, min(int(n), _INT_MAX))


def _addresses(device: torch.device, *wanted) -> list:
    """The addresses of contiguous tensors on `device`, given as (tensor, name, dtype, shape); raises for
    the first that is something else.  (A loop of plain comparisons: the smallest calls cost little more.)"""
    i = device.index if device.type == "cuda" else -1  # get_device() of a host tensor is -1
    out = []
    for t, name, dtype, shape in wanted:
        try:
            ok = t.dtype is dtype and t.get_device() == i and t.shape == shape and t.is_contiguous()
        except AttributeError:
            ok = False
        if not ok:
            _refuse(t, name, dtype, shape, device)
        out.append(t.data_ptr())
    return out


def _rows_of(t, name: str, dtype: torch.dtype, shape: Tuple[int, ...], device: torch.device) -> Tuple[int, int]:
    """(address, elements between rows) of a [rows, heads, dim] tensor whose heads are contiguous."""
    i = device.index if device.type == "cuda" else -1
    try:
        ok = t.dtype is dtype and t.get_device() == i and t.shape == shape
    except AttributeError:
        ok = False
    if not ok:
        _refuse(t, name, dtype, shape, device)
    rows, heads, dim = shape
    s0, s1, s2 = t.stride()
    if s2 == 1 and s1 == dim and (s0 >= heads * dim or rows <= 1):
        return t.data_ptr(), (s0 if rows > 1 else heads * dim)
    # sizes of one leave a stride without meaning
    if t.numel() and ((dim > 1 and s2 != 1) or (heads > 1 and s1 != dim) or (rows > 1 and s0 < heads * dim)):
        raise ValueError(f"{name}: the heads of a row must be contiguous and rows must not overlap, got strides {(s0, s1, s2)}")
    return t.data_ptr(), (s0 if rows > 1 else heads * dim)


_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


class _On:
    """Makes `device` and `stream` (None: the device's current one) current for the calls inside."""
    __slots__ = ("device", "stream", "ctx")

    def __init__(self, device: torch.device, stream: Optional[torch.cuda.Stream]):
        self.device, self.stream = device, stream

    def __enter__(self) -> int:
        if self.stream is not None:
            if self.stream.device != self.device:
                raise ValueError(f"stream: expected a stream of {self.device}, got one of {self.stream.device}")
            self.ctx = torch.cuda.stream(self.stream)  # also makes its device current
        else:
            self.ctx = torch.cuda.device(self.device)
        self.ctx.__enter__()
        return torch.cuda.current_stream(self.device).cuda_stream

    def __exit__(self, *a) -> None:
        self.ctx.__exit__(*a)


class _Here:
    """The same where the device is current and no stream is given: nothing to change."""
    __slots__ = ("raw",)

    def __init__(self, raw: int):
        self.raw = raw

    def __enter__(self) -> int:
        return self.raw

    def __exit__(self, *a) -> None:
        pass


def _on(device: torch.device, stream: Optional[torch.cuda.Stream]):
    i = device.index
    if stream is None and torch.cuda.current_device() == i:
        return _Here(_raw_stream(i) if _raw_stream else torch.cuda.current_stream(device).cuda_stream)
    return _On(device, stream)


def extend_tables(ctx_lens: torch.Tensor, new_rows: torch.Tensor, page_tables: torch.Tensor, free_pages: torch.Tensor,
                  free_begin: torch.Tensor, max_rows: int, out: Optional[RowPlan] = None, stream=None,
                  held_pages: Optional[torch.Tensor] = None) -> RowPlan:
    """Pages for the new rows of a batch and every new row's place.  ctx_lens, new_rows [nb];
    page_tables [nb, max_pages_per_seq], extended in place; free_pages [n] a stack of page ids taken
    from position free_begin [1] on.  Sequences are served in order while pages and max_rows last.
    `out`: a RowPlan to write into; its kv_lens may be ctx_lens and its free_end free_begin.
    `held_pages` [nb]: pages that each sequence has in its table, brought up to date in place; for
    sequences whose ctx_lens may go back (rejected rows), so that pages given for those rows are used
    again.  Without it a sequence holds the pages that its ctx_lens rows fill, and entries behind them
    are overwritten."""
    try:  # sizes first; _addresses holds every tensor to them
        dev, nb = ctx_lens.device, ctx_lens.shape[0]
        mpps, n_free = page_tables.shape[1], free_pages.shape[0]
        ok = dev.type == "cuda"
    except (AttributeError, IndexError):
        ok = False
    if not ok:
        _first(ctx_lens, "ctx_lens", 1), _first(page_tables, "page_tables", 2), _first(free_pages, "free_pages", 1)
    max_rows = int(max_rows)
    if not 0 <= max_rows <= _INT_MAX:
        raise ValueError("max_rows must be in [0, 2^31)")
    one, seqs, rows = (1,), (nb,), (max_rows,)
    with _on(dev, stream) as st:
        if out is None:
            def e(n):
                return torch.empty(n, dtype=_I32, device=dev)
            out = RowPlan(e(nb), e(nb + 1), e(max_rows), e(max_rows), e(max_rows), e(1))
        kv_lens, row_starts, row_seq, row_index, slots, free_end = out
        a_ctx, a_new, a_pt, a_free, a_begin, a_end, a_kv, a_rs, a_seq, a_idx, a_slots = _addresses(
            dev, (ctx_lens, "ctx_lens", _I32, seqs), (new_rows, "new_rows", _I32, seqs),
            (page_tables, "page_tables", _I32, (nb, mpps)), (free_pages, "free_pages", _I32, (n_free,)),
            (free_begin, "free_begin", _I32, one), (free_end, "out.free_end", _I32, one),
            (kv_lens, "out.kv_lens", _I32, seqs), (row_starts, "out.row_starts", _I32, (nb + 1,)),
            (row_seq, "out.row_seq", _I32, rows), (row_index, "out.row_index", _I32, rows), (slots, "out.slots", _I32, rows))
        a_held = 0 if held_pages is None else _addresses(dev, (held_pages, "held_pages", _I32, seqs))[0]
        # an empty tensor has no address, and the entry takes none that is null
        L.dflash_extend_tables_ex(a_ctx, a_new, _i32(nb, "sequences"), a_pt, _i32(mpps, "pages of a sequence"), a_free or a_pt,
                                  _i32(n_free, "free pages"), a_begin, a_end, a_kv, a_rs, a_seq or a_pt,
                                  a_idx or a_pt, a_slots or a_pt, max_rows, a_held, _status_word(dev).data_ptr(), st)
    return out


class PagedKV:
    """K/V pages of one layer: a tensor [pages, kv_heads, 2, 16 * head_dim] (bfloat16 or float32,
    contiguous but for the stride between pages), whose last dimension is a tile in the layout of
    dflash_kv_layout.  One layer of a larger tensor, or of a drafter's own pool
    (`Drafter.kv_pages`), is a view of it."""

    def __init__(self, pool: torch.Tensor):
        try:
            (P, nkv, two, tile), st = pool.shape, pool.stride()
            dtype, dev = pool.dtype, pool.device
            ok = dev.type == "cuda" and (dtype is _BF16 or dtype is _F32)
        except (AttributeError, ValueError):
            ok = False
        if not ok:
            _first(pool, "pool", 4, (_BF16, _F32))
        if two != 2 or (tile != 1024 and tile != 2048):
            raise ValueError(f"pool: expected shape [pages, kv_heads, 2, 16 * 64 or 16 * 128], got {tuple(pool.shape)}")
        if st[3] != 1 or st[2] != tile or (nkv > 1 and st[1] != 2 * tile):
            raise ValueError("pool: heads and tiles of a page must be contiguous")
        self.pool = pool
        self.head_dim = tile // 16
        self._c = L.dflash_kv_pages(pool.data_ptr(), st[0] if P > 1 else 2 * nkv * tile, _status_word(dev).data_ptr(),
                                    L.DFLASH_BF16 if dtype is _BF16 else L.DFLASH_F32, nkv, self.head_dim, P)
        self._workspace = None  # bytes that a call of attend needs

    @classmethod
    def empty(cls, num_pages: int, n_kv_heads: int, head_dim: int, dtype: torch.dtype = _BF16, device="cuda") -> "PagedKV":
        """A cache of its own (pages uninitialised: rows are defined once appended)."""
        return cls(torch.empty((num_pages, n_kv_heads, 2, 16 * head_dim), dtype=dtype, device=device))

    def append(self, k: torch.Tensor, v: torch.Tensor, slots: torch.Tensor, stream=None) -> torch.Tensor:
        """Rows k, v [n, kv_heads, head_dim] (any stride between rows) into slots [n] (negative: skipped)
        of the pages.  Returns the pages' tensor."""
        pool = self.pool
        dev = pool.device
        try:
            n = slots.shape[0]
        except (AttributeError, IndexError):
            _first(slots, "slots", 1)
            raise
        a_s, = _addresses(dev, (slots, "slots", _I32, (n,)))
        shape = (n, pool.shape[1], self.head_dim)
        a_k, ks = _rows_of(k, "k", pool.dtype, shape, dev)
        a_v, vs = _rows_of(v, "v", pool.dtype, shape, dev)
        with _on(dev, stream) as st:
            L.dflash_append_kv(self._c, a_k, ks, a_v, vs, a_s, _i32(n, "rows"), st)
        return pool

    def attend(self, q: torch.Tensor, page_tables: torch.Tensor, kv_lens: torch.Tensor, row_starts: torch.Tensor,
               max_new: int, causal: bool = True, window: int = 0, scale: Optional[float] = None,
               out: Optional[torch.Tensor] = None, lse: Optional[torch.Tensor] = None, stream=None):
        """Attention of each sequence's newest rows over its pages.  q [rows, heads, head_dim]; rows
        row_starts[s] .. row_starts[s + 1] - 1 are the last rows of sequence s, which has kv_lens[s].
        max_new: the longest chunk, or an upper bound (it picks the kernel).  scale: 1 / sqrt(head_dim)
        by default.  Returns out [rows, heads, head_dim] (a new one is zeroed, so that rows behind the
        last sequence hold zeros), or (out, lse) when `lse` [rows, heads] float32 is given."""
        pool = self.pool
        dev = pool.device
        hd = self.head_dim
        try:
            (n, nh, _), (nb, mpps) = q.shape, page_tables.shape
        except (AttributeError, ValueError):
            _first(q, "q", 3, (pool.dtype,)), _first(page_tables, "page_tables", 2)
            raise
        shape = (n, nh, hd)
        a_q, qs = _rows_of(q, "q", pool.dtype, shape, dev)
        a_pt, a_kv, a_rs = _addresses(dev, (page_tables, "page_tables", _I32, (nb, mpps)), (kv_lens, "kv_lens", _I32, (nb,)),
                                      (row_starts, "row_starts", _I32, (nb + 1,)))
        a_lse = 0 if lse is None else _addresses(dev, (lse, "lse", _F32, (n, nh)))[0]
        with _on(dev, stream) as st:
            if out is None:
                out = torch.zeros(shape, dtype=pool.dtype, device=dev)
            a_out, os_ = _rows_of(out, "out", pool.dtype, shape, dev)
            need = self._workspace
            if need is None:
                need = self._workspace = L.dflash_attend_workspace(self._c)
            ws = torch.empty(need, dtype=torch.uint8, device=dev) if need else None
            L.dflash_attend(self._c, a_q, qs, a_pt, _i32(mpps, "pages of a sequence"), a_kv, a_rs, _i32(nb, "sequences"),
                            _i32(n, "rows"), _limit(max_new), nh,
                            1.0 / math.sqrt(hd) if scale is None else float(scale), _limit(window), 1 if causal else 0,
                            a_out, os_, a_lse, ws.data_ptr() if need else 0, need, st)
        return out if lse is None else (out, lse)


def sample(logits: torch.Tensor, u: torch.Tensor, temperature: Optional[torch.Tensor] = None,
           top_k: Optional[torch.Tensor] = None, top_p: Optional[torch.Tensor] = None,
           min_p: Optional[torch.Tensor] = None, tokens: Optional[torch.Tensor] = None,
           probs: Optional[torch.Tensor] = None, stream=None):
    """One token per row of logits [rows, vocab] (bfloat16 or float32, any stride between rows) from
    uniform numbers u [rows] float32.  temperature, top_p, min_p float32 and top_k int32 [rows], each
    optional.  Returns tokens [rows] int32, or (tokens, probs) when `probs` [rows] float32 is given."""
    try:
        dev, dtype = logits.device, logits.dtype
        (rows, V), (st0, st1) = logits.shape, logits.stride()
        ok = dev.type == "cuda" and (dtype is _BF16 or dtype is _F32)
    except (AttributeError, ValueError):
        ok = False
    if not ok:
        _first(logits, "logits", 2, (_BF16, _F32))
    if (V > 1 and st1 != 1) or (rows > 1 and st0 < V):
        raise ValueError(f"logits: a row must be contiguous and rows must not overlap, got strides {(st0, st1)}")
    col = (rows,)
    given = [w for w in ((u, "u", _F32, col), (temperature, "temperature", _F32, col), (top_k, "top_k", _I32, col),
                         (top_p, "top_p", _F32, col), (min_p, "min_p", _F32, col), (probs, "probs", _F32, col),
                         (tokens, "tokens", _I32, col)) if w[0] is not None or w[1] == "u"]
    at = dict(zip((w[1] for w in given), _addresses(dev, *given)))
    with _on(dev, stream) as st:
        if tokens is None:
            tokens = torch.empty(rows, dtype=_I32, device=dev)
            at["tokens"] = tokens.data_ptr()
        get = at.get
        L.dflash_sample(logits.data_ptr(), st0 if rows > 1 else V, L.DFLASH_BF16 if dtype is _BF16 else L.DFLASH_F32, _i32(rows, "rows"),
                        _i32(V, "logits of a row"), at["u"], get("temperature", 0), get("top_k", 0), get("top_p", 0), get("min_p", 0), at["tokens"],
                        get("probs", 0), st)
    return tokens if probs is None else (tokens, probs)
