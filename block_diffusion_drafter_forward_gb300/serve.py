"""Serving operators around the drafter, over torch device tensors: page tables and row maps built
on the device (`extend_tables`), K/V rows appended to a paged cache and attended over (`PagedKV`; in
8 bits: `QuantKV`), trees of drafted tokens (`draft_tree`, `attend(tree=)`, `keep`), rotary positions
(`Rope`) and tokens drawn from logits (`sample`).  Thin calls of the C entries of the same names:
include/dflash.h states what each computes and refuses.

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

_I32, _I64, _F32, _BF16 = torch.int32, torch.int64, torch.float32, torch.bfloat16
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


class TreePlan(NamedTuple):
    """What `draft_tree` returns, for every layer's `attend` (device tensors)."""
    positions: torch.Tensor  # [rows] int32 position of each node: its sequence's context and its depth
    masks: torch.Tensor      # [rows, words] int64: bit j % 64 of word j // 64 is set for the node j itself and its ancestors


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
    i = device.index
    i = -1 if i is None else i  # get_device() of a host tensor is -1
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
    i = device.index
    i = -1 if i is None else i
    try:
        ok = t.dtype is dtype and t.get_device() == i and t.shape == shape
    except AttributeError:
        ok = False
    if not ok:
        _refuse(t, name, dtype, shape, device)
    rows, heads, dim = shape
    if t.is_contiguous():
        return t.data_ptr(), heads * dim
    s0, s1, s2 = t.stride()
    if s2 == 1 and s1 == dim and (s0 >= heads * dim or rows <= 1):
        return t.data_ptr(), (s0 if rows > 1 else heads * dim)
    # sizes of one leave a stride without meaning
    if t.numel() and ((dim > 1 and s2 != 1) or (heads > 1 and s1 != dim) or (rows > 1 and s0 < heads * dim)):
        raise ValueError(f"{name}: the heads of a row must be contiguous and rows must not overlap, got strides {(s0, s1, s2)}")
    return t.data_ptr(), (s0 if rows > 1 else heads * dim)


_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (lambda i: torch.cuda.current_stream(i).cuda_stream)
_device_now = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device


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
    if stream is None and _device_now() == i:
        return _Here(_raw_stream(i))
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


def draft_tree(parents: torch.Tensor, kv_lens: torch.Tensor, row_starts: torch.Tensor, max_nodes: int,
               out: Optional[TreePlan] = None, stream=None) -> TreePlan:
    """Positions and masks of drafted trees.  Rows row_starts[s] .. row_starts[s + 1] - 1 are the nodes of
    sequence s, its last rows of kv_lens[s]; parents [rows] is the node of the same sequence that a node
    follows (an earlier one), or -1 where it follows the context.  max_nodes: the largest tree, or a
    bound (at most 512); it sets the masks' words."""
    try:
        dev, n, nb = parents.device, parents.shape[0], kv_lens.shape[0]
        ok = dev.type == "cuda"
    except (AttributeError, IndexError):
        ok = False
    if not ok:
        _first(parents, "parents", 1), _first(kv_lens, "kv_lens", 1)
    max_nodes = int(max_nodes)
    if not 1 <= max_nodes <= 512:
        raise ValueError("max_nodes must be in [1, 512]")
    words = (max_nodes + 63) // 64
    if stream is not None or _device_now() != dev.index:
        with _On(dev, stream):
            return draft_tree(parents, kv_lens, row_starts, max_nodes, out)
    st = _raw_stream(dev.index)
    if out is None:
        out = TreePlan(torch.empty(n, dtype=_I32, device=dev), torch.empty((n, words), dtype=_I64, device=dev))
    positions, masks = out
    a_par, a_kv, a_rs, a_pos, a_mask = _addresses(
        dev, (parents, "parents", _I32, (n,)), (kv_lens, "kv_lens", _I32, (nb,)), (row_starts, "row_starts", _I32, (nb + 1,)),
        (positions, "out.positions", _I32, (n,)), (masks, "out.masks", _I64, (n, words)))
    rc = L.load().dflash_draft_tree(a_par, a_kv, a_rs, _i32(nb, "sequences"), _i32(n, "rows"), max_nodes, a_pos, a_mask,
                                    _status_word(dev).data_ptr(), st)
    if rc:
        L._check(rc, None)
    return out


class Rope:
    """Rotary positions with a table of frequencies on `device`: theta^(-2j / rotary_dim), divided by
    `linear`, or remapped by `yarn` = (factor, original length, beta fast, beta slow) as a drafter's
    configuration does.  Pairs are the halves of the rotated dims, or neighbours (interleaved).  `turns`
    [rotary_dim / 2] int64 holds the frequencies in 2^-64 turns per position; a model with others gives
    the attribute a tensor of its own, and `mscale` the factor of its rotated values."""

    def __init__(self, rotary_dim: int, theta: float = 1e6, linear: float = 1.0,
                 yarn: Optional[Tuple[float, float, float, float]] = None, interleaved: bool = False, device="cuda"):
        turns, self.mscale = L.dflash_rope_turns(int(rotary_dim), float(theta), float(linear), None if yarn is None else tuple(map(float, yarn)))
        self.rotary_dim, self.interleaved = int(rotary_dim), bool(interleaved)
        device = torch.device(device)
        if device.type == "cuda" and device.index is None:
            device = torch.device("cuda", torch.cuda.current_device())
        with torch.inference_mode(False):
            self.turns = torch.tensor(turns, dtype=_I64).to(device)  # (below 2^62)
        if device.type == "cuda":  # there for every stream
            torch.cuda.current_stream(device).synchronize()

    @property
    def turns(self) -> torch.Tensor:
        return self._turns

    @turns.setter
    def turns(self, t: torch.Tensor) -> None:
        if not isinstance(t, torch.Tensor):
            raise TypeError(f"turns: expected a torch.Tensor, got {type(t).__name__}")
        _addresses(t.device, (t, "turns", _I64, (self.rotary_dim // 2,)))
        self._turns, self._device = t, t.device

    def rotate(self, q: torch.Tensor, positions: torch.Tensor, k: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None,
               k_out: Optional[torch.Tensor] = None, inverse: bool = False, stream=None):
        """q [rows, heads, head_dim] and k [rows, kv_heads, head_dim] (any stride between rows) at `positions`
        [rows] int32, into `out` and `k_out` (new ones by default; an input itself: in place).  inverse: the
        map's transpose, which takes gradients back.  Returns out, or (out, k_out) when k is given."""
        try:
            n, nh, hd = q.shape
            dtype, dev = q.dtype, q.device
            ok = dev.type == "cuda" and (dtype is _BF16 or dtype is _F32)
        except (AttributeError, ValueError):
            ok = False
        if not ok:
            _first(q, "q", 3, (_BF16, _F32))
        turns = self._turns
        if self._device != dev:
            raise ValueError(f"q: the table is on {self._device}, got a tensor on {dev}")
        if turns.shape != (self.rotary_dim // 2,):  # (checked as it was given; changed since)
            _refuse(turns, "turns", _I64, (self.rotary_dim // 2,), dev)
        a_q, qs = _rows_of(q, "q", dtype, (n, nh, hd), dev)
        a_pos, = _addresses(dev, (positions, "positions", _I32, (n,)))
        a_k = ks = a_ko = kos = nk = 0
        if k is not None:
            if not isinstance(k, torch.Tensor) or k.dim() != 3:
                _first(k, "k", 3, (dtype,))
            nk = k.shape[1]
            a_k, ks = _rows_of(k, "k", dtype, (n, nk, hd), dev)
        elif k_out is not None:
            raise ValueError("k_out: given without k")
        if stream is not None or _device_now() != dev.index:
            with _On(dev, stream):
                return self.rotate(q, positions, k, out, k_out, inverse)
        st = _raw_stream(dev.index)
        if out is None:
            out = torch.empty((n, nh, hd), dtype=dtype, device=dev)
        a_o, os_ = _rows_of(out, "out", dtype, (n, nh, hd), dev)
        if k is not None:
            if k_out is None:
                k_out = torch.empty((n, nk, hd), dtype=dtype, device=dev)
            a_ko, kos = _rows_of(k_out, "k_out", dtype, (n, nk, hd), dev)
        rc = L.load().dflash_rotate(a_q, qs, a_o, os_, nh, a_k, ks, a_ko, kos, nk, L.DFLASH_BF16 if dtype is _BF16 else L.DFLASH_F32,
                                    _i32(n, "rows"), hd, self.rotary_dim, self.interleaved, inverse, a_pos, turns.data_ptr(),
                                    self.mscale, st)
        if rc:
            L._check(rc, None)
        return out if k is None else (out, k_out)


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
        self._rows = (dtype,)
        self._c = L.dflash_kv_pages(pool.data_ptr(), st[0] if P > 1 else 2 * nkv * tile, _status_word(dev).data_ptr(),
                                    L.DFLASH_BF16 if dtype is _BF16 else L.DFLASH_F32, nkv, self.head_dim, P)
        self._ref = ctypes.byref(self._c)
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
               out: Optional[torch.Tensor] = None, lse: Optional[torch.Tensor] = None, stream=None,
               tree: Optional[TreePlan] = None):
        """Attention of each sequence's newest rows over its pages.  q [rows, heads, head_dim]; rows
        row_starts[s] .. row_starts[s + 1] - 1 are the last rows of sequence s, which has kv_lens[s].
        max_new: the longest chunk, or an upper bound (it picks the kernel).  scale: 1 / sqrt(head_dim)
        by default.  tree: of `draft_tree` for these rows, whose nodes see the context and their own
        ancestors (`causal` is not looked at then, and a window is at least the masks' bits).  Returns out
        [rows, heads, head_dim] (a new one is zeroed, so that rows behind the last sequence hold zeros), or
        (out, lse) when `lse` [rows, heads] float32 is given."""
        dev = self.pool.device
        hd = self.head_dim
        try:
            (n, nh, _), (nb, mpps), dtype = q.shape, page_tables.shape, q.dtype
        except (AttributeError, ValueError):
            _first(q, "q", 3, self._rows), _first(page_tables, "page_tables", 2)
            raise
        if dtype not in self._rows:
            _first(q, "q", 3, self._rows)
        shape = (n, nh, hd)
        a_q, qs = _rows_of(q, "q", dtype, shape, dev)
        lens = ((page_tables, "page_tables", _I32, (nb, mpps)), (kv_lens, "kv_lens", _I32, (nb,)), (row_starts, "row_starts", _I32, (nb + 1,)))
        if lse is None:
            a_lse = 0
            a_pt, a_kv, a_rs = _addresses(dev, *lens)
        else:
            a_pt, a_kv, a_rs, a_lse = _addresses(dev, *lens, (lse, "lse", _F32, (n, nh)))
        a_pos = a_mask = words = 0
        if tree is not None:
            positions, masks = tree
            words = masks.shape[1] if isinstance(masks, torch.Tensor) and masks.dim() == 2 else 1
            a_pos, a_mask = _addresses(dev, (positions, "tree.positions", _I32, (n,)), (masks, "tree.masks", _I64, (n, words)))
            if not n:
                a_pos = a_mask = words = 0
        if stream is not None or _device_now() != dev.index:
            with _On(dev, stream):
                return self.attend(q, page_tables, kv_lens, row_starts, max_new, causal, window, scale, out, lse, tree=tree)
        st = _raw_stream(dev.index)
        if out is None:
            out = torch.zeros(shape, dtype=dtype, device=dev)
        a_out, os_ = _rows_of(out, "out", dtype, shape, dev)
        need = 0
        if dtype is _BF16:
            need = self._workspace
            if need is None:
                need = self._workspace = L.dflash_attend_workspace(self._c)
        ws = torch.empty(need, dtype=torch.uint8, device=dev) if need else None
        rc = L.load().dflash_attend_ex(
            self._ref, L.DFLASH_BF16 if dtype is _BF16 else L.DFLASH_F32, a_q, qs, a_pt, _i32(mpps, "pages of a sequence"),
            a_kv, a_rs, _i32(nb, "sequences"), _i32(n, "rows"), _limit(max_new), nh,
            1.0 / math.sqrt(hd) if scale is None else float(scale), _limit(window), 1 if causal else 0, a_mask or None, words,
            a_pos or None, a_out, os_, a_lse, ws.data_ptr() if need else 0, need, st)
        if rc:
            L._check(rc, None)
        return out if lse is None else (out, lse)

    def keep(self, page_tables: torch.Tensor, ctx_lens: torch.Tensor, path: torch.Tensor, path_lens: torch.Tensor,
             stream=None) -> torch.Tensor:
        """The rows of an accepted branch moved to where the sequence goes on: row ctx_lens[s] + path[s, i] to row
        ctx_lens[s] + i, i < path_lens[s].  path [nb, longest] rises within a sequence; its entries from
        path_lens[s] on are not read.  Returns the pages' tensor."""
        dev = self.pool.device
        try:
            (nb, mpps), (_, longest) = page_tables.shape, path.shape
        except (AttributeError, ValueError):
            _first(page_tables, "page_tables", 2), _first(path, "path", 2)
            raise
        a_pt, a_ctx, a_path, a_len = _addresses(
            dev, (page_tables, "page_tables", _I32, (nb, mpps)), (ctx_lens, "ctx_lens", _I32, (nb,)),
            (path, "path", _I32, (nb, longest)), (path_lens, "path_lens", _I32, (nb,)))
        if stream is not None or _device_now() != dev.index:
            with _On(dev, stream):
                return self.keep(page_tables, ctx_lens, path, path_lens)
        st = _raw_stream(dev.index)
        rc = L.load().dflash_keep_rows(self._ref, a_pt, _i32(mpps, "pages of a sequence"), a_ctx, _i32(nb, "sequences"), a_path,
                                       _i32(longest, "nodes of a path"), a_len, st)
        if rc:
            L._check(rc, None)
        return self.pool


class QuantKV(PagedKV):
    """The same in 8 bits: a uint8 tensor [pages, kv_heads, 32 * head_dim + 32] (contiguous but for the stride
    between pages) of e4m3 codes with a power of two for every row and head.  Rows are quantised as `append`
    writes them and are bf16 numbers from then on; `attend` takes bfloat16 or float32 queries."""

    def __init__(self, pool: torch.Tensor):
        try:
            (P, nkv, size), st = pool.shape, pool.stride()
            dev = pool.device
            ok = dev.type == "cuda" and pool.dtype is torch.uint8
        except (AttributeError, ValueError):
            ok = False
        if not ok:
            _first(pool, "pool", 3, (torch.uint8,))
        if size != 32 * 64 + 32 and size != 32 * 128 + 32:
            raise ValueError(f"pool: expected shape [pages, kv_heads, 32 * 64 + 32 or 32 * 128 + 32], got {tuple(pool.shape)}")
        if st[2] != 1 or (nkv > 1 and st[1] != size):
            raise ValueError("pool: heads of a page must be contiguous")
        self.pool = pool
        self.head_dim = (size - 32) // 32
        self._rows = (_BF16, _F32)
        self._c = L.dflash_kv_pages(pool.data_ptr(), st[0] if P > 1 else nkv * size, _status_word(dev).data_ptr(),
                                    L.DFLASH_FP8E4M3_ROWEXP, nkv, self.head_dim, P)
        self._ref = ctypes.byref(self._c)
        self._workspace = None

    @classmethod
    def empty(cls, num_pages: int, n_kv_heads: int, head_dim: int, device="cuda") -> "QuantKV":
        """A cache of its own (pages uninitialised: rows are defined once appended)."""
        return cls(torch.empty((num_pages, n_kv_heads, 32 * head_dim + 32), dtype=torch.uint8, device=device))

    def append(self, k: torch.Tensor, v: torch.Tensor, slots: torch.Tensor, stream=None) -> torch.Tensor:
        """Rows k, v [n, kv_heads, head_dim] (bfloat16 or float32, any stride between rows), quantised, into slots [n]
        (negative: skipped; one named twice holds nothing meaningful) of the pages.  Returns the pages' tensor."""
        dev = self.pool.device
        try:
            n, dtype = slots.shape[0], k.dtype
        except (AttributeError, IndexError):
            _first(slots, "slots", 1), _first(k, "k", 3, self._rows)
            raise
        if dtype not in self._rows:
            _first(k, "k", 3, self._rows)
        a_s, = _addresses(dev, (slots, "slots", _I32, (n,)))
        shape = (n, self.pool.shape[1], self.head_dim)
        a_k, ks = _rows_of(k, "k", dtype, shape, dev)
        a_v, vs = _rows_of(v, "v", dtype, shape, dev)
        if stream is not None or _device_now() != dev.index:
            with _On(dev, stream):
                return self.append(k, v, slots)
        st = _raw_stream(dev.index)
        rc = L.load().dflash_append_kv_quant(self._ref, L.DFLASH_BF16 if dtype is _BF16 else L.DFLASH_F32, a_k, ks, a_v, vs, a_s,
                                             _i32(n, "rows"), st)
        if rc:
            L._check(rc, None)
        return self.pool

    def read(self, slots: torch.Tensor, dtype: torch.dtype = _BF16, k: Optional[torch.Tensor] = None,
             v: Optional[torch.Tensor] = None, stream=None) -> Tuple[torch.Tensor, torch.Tensor]:
        """(k, v) [n, kv_heads, head_dim]: the rows in slots [n] as numbers (zeros where a slot is negative), exact
        in either dtype.  k, v: tensors to write into."""
        dev = self.pool.device
        if dtype not in self._rows:
            raise ValueError(f"dtype: expected {' or '.join(map(str, self._rows))}, got {dtype}")
        try:
            n = slots.shape[0]
        except (AttributeError, IndexError):
            _first(slots, "slots", 1)
            raise
        a_s, = _addresses(dev, (slots, "slots", _I32, (n,)))
        shape = (n, self.pool.shape[1], self.head_dim)
        if stream is not None or _device_now() != dev.index:
            with _On(dev, stream):
                return self.read(slots, dtype, k, v)
        st = _raw_stream(dev.index)
        if k is None:
            k = torch.empty(shape, dtype=dtype, device=dev)
        if v is None:
            v = torch.empty(shape, dtype=dtype, device=dev)
        a_k, ks = _rows_of(k, "k", dtype, shape, dev)
        a_v, vs = _rows_of(v, "v", dtype, shape, dev)
        rc = L.load().dflash_read_kv_quant(self._ref, L.DFLASH_BF16 if dtype is _BF16 else L.DFLASH_F32, a_s, _i32(n, "rows"),
                                           a_k, ks, a_v, vs, st)
        if rc:
            L._check(rc, None)
        return k, v


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
