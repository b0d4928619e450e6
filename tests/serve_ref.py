"""Plain 64-bit forms of the serving operators for their tests: loops over sequences and rows, from
the definitions in include/dflash.h."""
import math

import numpy as np
import torch

PAGE = 16


def tables(ctx, new, table, free, begin, max_rows):
    """(table, kv_lens, row_starts, row_seq, row_index, slots, free_end) as int lists/arrays."""
    table = np.array(table.tolist() if isinstance(table, torch.Tensor) else table, dtype=np.int64)
    nb, mpps = table.shape
    seq, idx, slot, kv, starts = [], [], [], [], [0]
    at, rows, room = begin, 0, True
    want_pages = begin
    for s in range(nb):
        c, n = int(ctx[s]), int(new[s])
        if c < 0 or n < 0 or c + n > mpps * PAGE:
            n_ok, need = 0, 0
        else:
            n_ok, need = n, -(-(c + n) // PAGE) - (-(-c // PAGE))
        rows += n_ok
        want_pages += need
        if want_pages > len(free) or rows > max_rows or begin < 0:
            room = False
        if not room:
            n_ok = need = 0
        held = -(-c // PAGE)
        for i in range(need):
            table[s, held + i] = free[at + i]
        at += need
        for i in range(n_ok):
            j = c + i
            page = int(table[s, j // PAGE])
            seq.append(s), idx.append(j), slot.append(page * PAGE + j % PAGE if page >= 0 else -1)
        kv.append(c + n_ok)
        starts.append(starts[-1] + n_ok)
    pad = [-1] * (max_rows - len(seq))
    return table, kv, starts, seq + pad, idx + pad, slot + pad, [at]


def k_off(j, d, hd):
    return ((j // 8) * (hd // 8) + d // 8) * 64 + (j % 8) * 8 + d % 8


def v_off(j, d):
    return ((d // 8) * 2 + j // 8) * 64 + (d % 8) * 8 + j % 8


def put(pool, k, v, slots):
    """The pages [P, nkv, 2, 16 hd] after rows k, v [n, nkv, hd] went to `slots` (a copy)."""
    pool = pool.clone()
    hd = k.shape[2]
    d = torch.arange(hd)
    for i, s in enumerate(int(x) for x in slots):
        if s < 0 or s >= pool.shape[0] * PAGE:
            continue
        pool[s // PAGE, :, 0, k_off(s % PAGE, d, hd)] = k[i]
        pool[s // PAGE, :, 1, v_off(s % PAGE, d)] = v[i]
    return pool


def rows_of(pool, table_row, n):
    """K and V [n, nkv, hd] of a sequence's rows, in 64 bits."""
    hd = pool.shape[3] // PAGE
    d = torch.arange(hd, device=pool.device)
    j = torch.arange(n, device=pool.device)
    pages = table_row[: -(-n // PAGE)].long()[j // PAGE] if n else j
    j = (j % PAGE)[:, None]
    kk = pool[pages, :, 0].gather(2, k_off(j, d, hd)[:, None].expand(-1, pool.shape[1], -1)) if n else pool.new_zeros(0, pool.shape[1], hd)
    vv = pool[pages, :, 1].gather(2, v_off(j, d[None])[:, None].expand(-1, pool.shape[1], -1)) if n else kk
    return kk.double(), vv.double()


def attend(q, pool, table, kv_lens, starts, causal, window, scale):
    """(out, lse, spread, dots) in 64 bits for the rows of the sequences (0 elsewhere): spread =
    sum_j p_j |v_j|, dots = max_j sum_d |q_d k_jd|, for tolerances."""
    n_rows, nh, hd = q.shape
    out = torch.zeros(n_rows, nh, hd, dtype=torch.float64, device=q.device)
    spread, lse = torch.zeros_like(out), torch.zeros(n_rows, nh, dtype=torch.float64, device=q.device)
    dots = torch.zeros_like(lse)
    for s in range(len(kv_lens)):
        a, n, kv = starts[s], starts[s + 1] - starts[s], kv_lens[s]
        if not n:
            continue
        K, V = rows_of(pool, table[s], kv)
        g = nh // K.shape[1]
        K, V = K.repeat_interleave(g, 1), V.repeat_interleave(g, 1)
        qs = q[a:a + n].double()
        sc = torch.einsum("ihd,jhd->hij", qs, K) * scale
        pos = (kv - n + torch.arange(n, device=q.device))[:, None]
        key = torch.arange(kv, device=q.device)[None]
        hide = torch.zeros(n, kv, dtype=torch.bool, device=q.device)
        if causal:
            hide |= key > pos
        if window > 0:
            hide |= pos - key >= window
        sc = sc.masked_fill(hide, -math.inf)
        l = torch.logsumexp(sc, 2) if kv else torch.full((nh, n), -math.inf, dtype=torch.float64, device=q.device)
        p = torch.exp(sc - torch.where(l > -math.inf, l, 0.0)[..., None])
        out[a:a + n] = torch.einsum("hij,jhd->ihd", p, V)
        spread[a:a + n] = torch.einsum("hij,jhd->ihd", p, V.abs())
        lse[a:a + n] = l.t()
        if kv:
            dots[a:a + n] = (torch.einsum("ihd,jhd->hij", qs.abs(), K.abs()) * scale).amax(2).t()
    return out, lse, spread, dots


def sample(x, u, T=1.0, k=0, p=1.0, lo=0.0):
    """(token, probability) of one row of logits (a float64 numpy array)."""
    x = np.where(np.isnan(x), -np.inf, x)
    m = x.max() if x.size else -np.inf
    if m == -np.inf or not (0 <= T < np.inf):
        return -1, 0.0
    if T == 0:
        return int(np.argmax(x)), 1.0
    with np.errstate(invalid="ignore", over="ignore"):
        w = np.where(x == m, 1.0, np.exp((x - m) / T))
    w[~(w >= 2.0 ** -40)] = 0.0
    order = np.lexsort((np.arange(x.size), -x))
    order = order[x[order] > -np.inf]
    if k > 0:
        order = order[:k]
    if p < 1:
        ws = w[order]
        before = np.cumsum(ws) - ws
        keep = before < max(p, 0.0) * ws.sum()
        keep[0] = True
        order = order[keep]
    order = np.sort(order[w[order] >= lo])
    ws = w[order]
    if not ws.size or ws.sum() == 0:
        return -1, 0.0
    c = np.cumsum(ws)
    u = u if u > 0 else 0.0
    i = int(np.searchsorted(c, u * c[-1], side="right"))
    i = min(i, int(np.flatnonzero(ws)[-1]))
    return int(order[i]), float(ws[i] / c[-1])
