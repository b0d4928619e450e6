"""Plain 64-bit forms of the operators that verify drafted trees, of rotary positions and of pages in 8
bits, for their tests: loops and index arithmetic from the definitions in include/dflash.h."""
import math

import torch

import serve_ref as R

PAGE = 16


# ------------------------------------------------------------------------------ rotary positions
def inv_freq(rd, theta, linear=1.0, yarn=None):
    """(angles of one position, mscale), as Python floats."""
    base = [theta ** (-2.0 * j / rd) / linear for j in range(rd // 2)]
    if yarn is None:
        return base, 1.0
    factor, orig, fast, slow = yarn
    edge = [rd * math.log(orig / (b * 2 * math.pi)) / (2 * math.log(theta)) for b in (fast, slow)]
    low, high = max(math.floor(edge[0]), 0), min(math.ceil(edge[1]), rd - 1)
    span = high - low if high != low else 0.001
    out = []
    for j, f in enumerate(base):
        keep = 1 - min(max((j - low) / span, 0.0), 1.0)
        out.append(f * keep + f / factor * (1 - keep))
    return out, 0.1 * math.log(factor) + 1


def rotate(x, positions, turns, mscale, interleaved, inverse=False):
    """x [rows, heads, hd] float64 by the table's own whole numbers; and the sum of the two magnitudes that
    meet in each output."""
    rd = 2 * len(turns)
    angle = torch.tensor([[(p * t % 2 ** 64) / 2 ** 64 * 2 * math.pi for t in turns] for p in positions.tolist()],
                         dtype=torch.float64, device=x.device).view(len(positions), rd // 2)
    c, s = torch.cos(angle)[:, None] * mscale, torch.sin(angle)[:, None] * (-mscale if inverse else mscale)
    y, size = x.clone(), x.abs()
    a, b = (slice(0, rd, 2), slice(1, rd, 2)) if interleaved else (slice(0, rd // 2), slice(rd // 2, rd))
    y[..., a] = x[..., a] * c - x[..., b] * s
    y[..., b] = x[..., b] * c + x[..., a] * s
    size[..., a] = size[..., b] = (x[..., a].abs() + x[..., b].abs()) * mscale
    size[..., rd:] = 0
    return y, size


# ------------------------------------------------------------------------------ trees
def tree(parents):
    """(depths, [n][n] lists of truth values: which nodes a node sees) of one tree."""
    depth, see = [], []
    for i, p in enumerate(parents):
        row = list(see[p]) if p >= 0 else [False] * len(parents)
        row[i] = True
        see.append(row)
        depth.append(depth[p] + 1 if p >= 0 else 0)
    return depth, see


def words(see, n_words):
    """The masks of one tree as int64 numbers."""
    out = []
    for row in see:
        bits = sum(1 << j for j, x in enumerate(row) if x)
        w = [(bits >> 64 * k) & (2 ** 64 - 1) for k in range(n_words)]
        out.append([x - 2 ** 64 if x >= 2 ** 63 else x for x in w])
    return out


# ------------------------------------------------------------------------------ pages in 8 bits
def k8(j, d):
    return (d // 64) * 1024 + j * 64 + ((d // 16 % 4) ^ (j // 2 % 4)) * 16 + d % 16


def v8(j, d):
    return (d // 32) * 512 + (d % 8) * 64 + ((j // 4) ^ (d % 8 // 2)) * 16 + (d % 32 // 8) * 4 + j % 4


def code_value(c):
    """An e4m3 code as a number."""
    e, m = c >> 3 & 15, c & 7
    if e == 15 and m == 7:
        return math.nan
    v = m / 8 * 2.0 ** -6 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7)
    return -v if c & 128 else v


_VALUES = torch.tensor([code_value(c) for c in range(256)], dtype=torch.float64)


def quantise(x):
    """(values that the codes of rows x [..., hd] stand for, exponent bytes), float64 / int64."""
    x = x.double()
    fine = torch.isfinite(x)
    top = torch.where(fine, x.abs(), 0.0).amax(-1)
    k = torch.full_like(top, -118)
    for e in range(119, -119, -1):  # the smallest that holds the largest
        k = torch.where(top <= 448 * 2.0 ** e, e, k)
    k = torch.where(top > 448 * 2.0 ** 119, 119, k)
    unit = torch.pow(torch.tensor(2.0, dtype=torch.float64), k)[..., None]
    y = torch.where(fine, x / unit, 0.0).clamp(-448, 448)
    e = torch.floor(torch.log2(y.abs().clamp(min=2.0 ** -6)))
    e = torch.where(y.abs() >= torch.pow(2.0, e + 1), e + 1, torch.where(y.abs() < torch.pow(2.0, e), e - 1, e)).clamp(min=-6)
    step = torch.pow(torch.tensor(2.0, dtype=torch.float64), e - 3)
    y = torch.round(y / step) * step * unit
    return torch.where(fine, y, math.nan), (k + 127).long()


def rows8(pool, table_row, n):
    """K and V [n, nkv, hd] of a sequence's rows, in 64 bits."""
    pool = pool.cpu()
    nkv, hd = pool.shape[1], (pool.shape[2] - 32) // 32
    d, j = torch.arange(hd), torch.arange(n)
    page = table_row.cpu().long()[j // PAGE] if n else j
    j = (j % PAGE)[:, None]
    out = []
    for side, off in ((0, k8(j, d[None])), (1, v8(j, d[None]))):
        at = (off + side * 16 * hd)[:, None].expand(-1, nkv, -1)
        codes = pool[page].gather(2, at).long()
        e = pool[page][:, :, 32 * hd + 16 * side:32 * hd + 16 * side + 16].gather(2, j[:, None].expand(-1, nkv, 1)).double()
        out.append(_VALUES[codes] * torch.pow(2.0, e - 127))
    return out


def put8(pool, k, v, slots):
    """The pages after rows k, v [n, nkv, hd] went to `slots` (a copy): the bytes that the definition gives.
    NaN keeps the sign bit out: code 127."""
    pool = pool.clone()
    hd = k.shape[2]
    d = torch.arange(hd)
    by_value = {}
    for c in range(255, -1, -1):
        by_value[code_value(c) if c & 127 else (c, 0)] = c
    for side, x in ((0, k), (1, v)):
        y, e = quantise(x)
        unit = torch.pow(torch.tensor(2.0, dtype=torch.float64), e.double() - 127)[..., None]
        z = y / unit
        for i, s in enumerate(int(t) for t in slots):
            if s < 0 or s >= pool.shape[0] * PAGE:
                continue
            for h in range(k.shape[1]):
                codes = []
                for a, orig in zip(z[i, h].tolist(), x[i, h].tolist()):
                    if math.isnan(a):
                        codes.append(127)
                    elif a == 0:
                        codes.append(128 if math.copysign(1, orig) < 0 else 0)
                    else:
                        codes.append(by_value[a])
                off = k8(s % PAGE, d) if side == 0 else v8(s % PAGE, d)
                pool[s // PAGE, h, side * 16 * hd + off] = torch.tensor(codes, dtype=torch.uint8)
                pool[s // PAGE, h, 32 * hd + 16 * side + s % PAGE] = int(e[i, h])
    return pool


# ------------------------------------------------------------------------------ attention
def attend(q, rows, lens, starts, scale, causal=True, window=0, parents=None):
    """(out, lse, spread, dots) as serve_ref.attend gives them; rows(s, n): K and V of sequence s; parents: of
    every row, for trees."""
    n_rows, nh, hd = q.shape
    dev = q.device
    out = torch.zeros(n_rows, nh, hd, dtype=torch.float64, device=dev)
    spread, lse = torch.zeros_like(out), torch.zeros(n_rows, nh, dtype=torch.float64, device=dev)
    dots = torch.zeros_like(lse)
    for s in range(len(lens)):
        a, n, kv = starts[s], starts[s + 1] - starts[s], lens[s]
        if not n:
            continue
        K, V = (x.to(dev) for x in rows(s, kv))
        g = nh // K.shape[1]
        K, V = K.repeat_interleave(g, 1), V.repeat_interleave(g, 1)
        qs = q[a:a + n].double()
        ctx = kv - n
        key = torch.arange(kv, device=dev)[None]
        if parents is None:
            pos = (ctx + torch.arange(n, device=dev))[:, None]
            hide = key > pos if causal else torch.zeros(n, kv, dtype=torch.bool, device=dev)
            if window > 0:
                hide = hide | (pos - key >= window)
        else:
            depth, see = tree(parents[a:a + n])
            pos = (ctx + torch.tensor(depth, device=dev))[:, None]
            hide = (pos - key >= window) if window > 0 else torch.zeros(n, kv, dtype=torch.bool, device=dev)
            hide[:, ctx:] = ~torch.tensor(see, device=dev)
        sc = (torch.einsum("ihd,jhd->hij", qs, K) * scale).masked_fill(hide, -math.inf)
        l = torch.logsumexp(sc, 2) if kv else torch.full((nh, n), -math.inf, dtype=torch.float64, device=dev)
        p = torch.exp(sc - torch.where(l > -math.inf, l, 0.0)[..., None])
        out[a:a + n] = torch.einsum("hij,jhd->ihd", p, V)
        spread[a:a + n] = torch.einsum("hij,jhd->ihd", p, V.abs())
        lse[a:a + n] = l.t()
        if kv:
            dots[a:a + n] = (torch.einsum("ihd,jhd->hij", qs.abs(), K.abs()) * scale).masked_fill(hide, 0.0).amax(2).t()
    return out, lse, spread, dots


def rows16(pool, table):
    return lambda s, n: R.rows_of(pool, table[s], n)
