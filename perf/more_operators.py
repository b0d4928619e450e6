"""Cases of the operators that a target model calls when it verifies drafted tokens over a paged cache:
positions into queries and keys, trees of drafted tokens, and a cache held in 8 bits.

  rotate   Rope.rotate: rotary positions of a step's queries and keys (half or interleaved pairs, all
           of a head or part of it, plain, linear or YaRN frequencies)
  tree     draft_tree and PagedKV.attend(tree=): positions and masks of a batch of drafted trees, and
           their attention over the paged rows and over their own ancestors
  keep     PagedKV.keep: the rows of an accepted branch moved to where the sequence goes on
  store8   QuantKV.append and QuantKV.read: K and V rows quantised as they are written (e4m3 codes and a
           power of two per row and head), and read back
  attend8  QuantKV.attend: single tokens, blocks, trees and prompts over such a cache

`run` computes an operator in plain torch operations, or (own = True) through the package's entry
points.  Lengths are a function of the case alone; values, page ids and trees of the seed.
"""
import math
import random

import torch

own = False
PAGE = 16
_ropes = {}


# ------------------------------------------------------------------------------------- cases
def listed():
    return [
        # one token of 64 sequences on the 8-layer drafter's heads: a decode step's smallest kernel
        dict(name="rotate_step_64", op="rotate", rows=64, nh=32, nkv=4, hd=128, rd=128, interleaved=False, scaling="plain",
             theta=1e6, far=8192, dtype="bf16"),
        # a prefill step of 16 Ki rows on the wide drafter's heads, YaRN frequencies
        dict(name="rotate_prompt_16384", op="rotate", rows=16384, nh=64, nkv=8, hd=128, rd=128, interleaved=False,
             scaling="yarn", theta=1e6, far=262144, dtype="bf16"),
        # one sequence verifying a tree of 32 nodes at the benchmark's context: latency
        dict(name="tree_1x32", op="tree", nb=1, new_lo=32, new_hi=32, ctx_lo=4096, ctx_hi=4096, nh=32, nkv=4, hd=128, window=0),
        # the benchmark's ragged batch, trees of 33 to 64 nodes
        dict(name="tree_32x64", op="tree", nb=32, new_lo=33, new_hi=64, ctx_lo=512, ctx_hi=8192, nh=32, nkv=4, hd=128, window=0),
        # the accepted branch of one tree, one layer
        dict(name="keep_1x32", op="keep", nb=1, new_lo=32, new_hi=32, ctx_lo=300, ctx_hi=300, nkv=4, hd=128, dtype="bf16"),
        # the accepted branches of a large batch of trees, the wide drafter's K/V heads
        dict(name="keep_256x64", op="keep", nb=256, new_lo=33, new_hi=64, ctx_lo=0, ctx_hi=200, nkv=8, hd=128, dtype="bf16"),
        # K/V of a verification step (64 sequences x 16 rows) into the 8-bit cache and back
        dict(name="store8_verify_64x16", op="store8", nb=64, new_lo=16, new_hi=16, ctx_lo=0, ctx_hi=500, nkv=4, hd=128, dtype="bf16"),
        # K/V of a prefill step: ragged prompts of 16 Ki rows together, 8 K/V heads
        dict(name="store8_prompts_24", op="store8", nb=24, new_lo=33, new_hi=1333, ctx_lo=0, ctx_hi=700, nkv=8, hd=128, dtype="bf16"),
        # one sequence decoding one token at the benchmark's context: latency
        dict(name="attend8_decode_1x4096", op="attend8", nb=1, new_lo=1, new_hi=1, ctx_lo=4096, ctx_hi=4096, nh=32, nkv=4, hd=128,
             window=0, tree=False),
        # long-context decoding, the wide drafter's heads: what an 8-bit cache is for
        dict(name="attend8_decode_16x32768", op="attend8", nb=16, new_lo=1, new_hi=1, ctx_lo=16001, ctx_hi=32767, nh=64, nkv=8,
             hd=128, window=0, tree=False),
        # the benchmark's ragged batch, every sequence verifying a block of 16 tokens
        dict(name="attend8_verify_32x16", op="attend8", nb=32, new_lo=16, new_hi=16, ctx_lo=512, ctx_hi=8192, nh=32, nkv=4, hd=128,
             window=0, tree=False),
        # one long prompt in one chunk
        dict(name="attend8_prompt_8192", op="attend8", nb=1, new_lo=8192, new_hi=8192, ctx_lo=0, ctx_hi=0, nh=32, nkv=4, hd=128,
             window=0, tree=False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("rotate", "tree", "tree", "keep", "store8", "attend8", "attend8"))
    if op == "rotate":
        nkv, hd = rng.choice((1, 2, 4, 8)), rng.choice((64, 128))
        return dict(op=op, rows=_log(rng, 1, 16384), nh=nkv * rng.choice((1, 4, 5, 8)), nkv=nkv, hd=hd,
                    rd=rng.choice((hd, hd, hd // 2, 48, 32)), interleaved=rng.random() < 0.5,
                    scaling=rng.choice(("plain", "linear", "yarn")), theta=rng.choice((1e4, 5e5, 1e6)),
                    far=_log(rng, 100, 1000000), dtype=rng.choice(("bf16", "f32")))
    if op in ("keep", "store8"):
        hd = rng.choice((64, 128))
        nb = _log(rng, 1, 64 if op == "store8" else 256)
        lo = rng.choice((0, 1))
        most = max(1, 16384 // nb) if op == "store8" else 255
        return dict(op=op, nb=nb, new_lo=lo, new_hi=lo + _log(rng, 1, most), ctx_lo=0, ctx_hi=_log(rng, 16, 500),
                    nkv=rng.choice((1, 2, 4, 8)), hd=hd, dtype=rng.choice(("bf16", "f32")))
    nkv, group, hd = rng.choice((1, 2, 4, 8)), rng.choice((1, 4, 5, 8, 16)), rng.choice((64, 128))
    case = dict(op=op, nkv=nkv, nh=nkv * min(group, 64 // nkv), hd=hd, window=rng.choice((0, 0, _log(rng, 256, 4096))))
    form = rng.choice(("tree", "single", "single", "block", "prompt")) if op == "attend8" else "tree"
    if op == "attend8":
        case["tree"] = form == "tree"
    if form == "tree":
        lo = rng.choice((0, 1, 1))
        nb = _log(rng, 1, 32)
        new = lo + _log(rng, 2, 255)
        hi = _log(rng, 16, max(64, min(8192, 32 * 64 * 8192 // (nb * new))))
        return dict(case, nb=nb, new_lo=lo, new_hi=new, ctx_lo=hi // 4, ctx_hi=hi)
    if form == "single":
        nb = _log(rng, 1, 64)
        hi = _log(rng, 64, min(32768, 262144 // nb))
        return dict(case, nb=nb, new_lo=1, new_hi=1, ctx_lo=hi // 2, ctx_hi=hi)
    if form == "block":
        nb = _log(rng, 1, 32)
        hi = _log(rng, 64, 8192)
        return dict(case, nb=nb, new_lo=1, new_hi=rng.randint(2, 16), ctx_lo=hi // 4, ctx_hi=hi)
    return dict(case, nb=rng.randint(1, 6), new_lo=0, new_hi=_log(rng, 17, 1500), ctx_lo=0, ctx_hi=_log(rng, 16, 2500))


def _lens(case):
    """Context rows and new rows of every sequence (a function of the case alone)."""
    r = random.Random("lens %(nb)d %(new_lo)d %(new_hi)d %(ctx_lo)d %(ctx_hi)d" % case)
    ctx = [r.randint(case["ctx_lo"], case["ctx_hi"]) for _ in range(case["nb"])]
    new = [r.randint(case["new_lo"], case["new_hi"]) for _ in range(case["nb"])]
    if not any(new):
        new[0] = case["new_hi"]
    return ctx, new


def _up(a, b):
    return -(-a // b)


def _starts(new):
    out = [0]
    for n in new:
        out.append(out[-1] + n)
    return out


# ------------------------------------------------------------------------------------- inputs
def _i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _dtype(case):
    return torch.float32 if case.get("dtype") == "f32" else torch.bfloat16


def _yarn(case):
    return (32.0, 8192.0, 32.0, 1.0) if case["scaling"] == "yarn" else None


def _inv_freq(case):
    """(angle of one position for every pair, float64, and the scale of the rotated values)."""
    r, theta = case["rd"], case["theta"]
    j = torch.arange(r // 2, dtype=torch.float64)
    base = theta ** (-2.0 * j / r)
    if case["scaling"] == "linear":
        return base / 4.0, 1.0
    if case["scaling"] == "plain":
        return base, 1.0
    factor, orig, fast, slow = _yarn(case)
    edge = lambda beta: r * math.log(orig / (beta * 2 * math.pi)) / (2 * math.log(theta))  # noqa: E731
    low, high = max(math.floor(edge(fast)), 0.0), min(math.ceil(edge(slow)), r - 1.0)
    ramp = ((j - low) / (high - low if abs(high - low) >= 1e-6 else high - low + 0.001)).clamp(0.0, 1.0)
    return base / factor * ramp + base * (1 - ramp), 0.1 * math.log(factor) + 1.0


def _parents(new, seed):
    """A tree of every sequence's rows: node i hangs on one of the few nodes before it, or on the context."""
    r = random.Random("tree %d" % seed)
    return [[-1 if i == 0 or r.random() < 0.03 else r.randint(max(0, i - 1 - r.choice((0, 0, 3, 9))), i - 1) for i in range(n)] for n in new]


def _offsets(hd, es):
    """Element offsets [16, hd] of a page's rows in a head's K tile and V tile, bf16 / fp32 (es > 1) or 8 bits."""
    j, d = torch.arange(PAGE)[:, None], torch.arange(hd)[None]
    if es > 1:
        return (j // 8 * (hd // 8) + d // 8) * 64 + j % 8 * 8 + d % 8, (d // 8 * 2 + j // 8) * 64 + d % 8 * 8 + j % 8
    k = d // 64 * 1024 + j * 64 + ((d // 16 % 4) ^ (j // 2 % 4)) * 16 + d % 16
    return k, d // 32 * 512 + d % 8 * 64 + ((j // 4) ^ (d % 8 // 2)) * 16 + d % 32 // 8 * 4 + j % 4


def _pow2(k):
    """2^k in 32 bits, by its exponent's bits (infinity for 128)."""
    return ((k.to(torch.int32) + 127) << 23).view(torch.float32)


def _quantised(x):
    """(e4m3 codes as bytes, exponent bytes) of rows [..., hd]: the codes of x / 2^k, k the smallest with
    max |x| <= 448 2^k (kept in [-118, 119]), the byte k + 127."""
    top = x.abs().amax(-1).float()
    f, e = torch.frexp(top)
    k = torch.where(top > 0, e - torch.where(f <= 0.875, 9, 8), -118).clamp(-118, 119)
    codes = (x.float() * _pow2(-k)[..., None]).clamp(-448.0, 448.0).to(torch.float8_e4m3fn).view(torch.uint8)
    return codes, (k + 127).to(torch.uint8)


def _pages(case, g):
    """Page tables of a shared pool: each sequence's pages are a run of one random permutation."""
    ctx, new = _lens(case)
    pages = [_up(c + n, PAGE) for c, n in zip(ctx, new)]
    mpps, total = max(max(pages), 1) + 2, sum(pages) + 3
    perm = torch.randperm(total, generator=g).to(torch.int32)
    table = torch.full((case["nb"], mpps), -1, dtype=torch.int32)
    at = 0
    for s, n in enumerate(pages):
        table[s, :n] = perm[at:at + n]
        at += n
    return ctx, new, total, table


def _behind(ctx, new, table, total):
    """[pages, 16]: rows that no sequence has written (part-full last pages)."""
    ends = torch.full((total,), PAGE, dtype=torch.int64)
    for s, (c, n) in enumerate(zip(ctx, new)):
        if (c + n) % PAGE:
            ends[int(table[s, (c + n) // PAGE])] = (c + n) % PAGE
    return (torch.arange(PAGE)[None] >= ends[:, None]).cuda()


def _pool16(case, total, behind, gd):
    """Pages of unit keys and values; rows that were never written hold NaN."""
    nkv, hd, dt = case["nkv"], case["hd"], _dtype(case)
    pool = torch.randn((total, nkv, 2, PAGE * hd), generator=gd, device="cuda").to(dt)
    ko, vo = _offsets(hd, 2)
    for side, off in ((0, ko), (1, vo)):
        row = torch.empty(PAGE * hd, dtype=torch.int64)
        row[off.reshape(-1)] = torch.arange(PAGE).repeat_interleave(hd)
        pool[:, :, side].masked_fill_(behind[:, row.cuda()][:, None], float("nan"))
    return pool


def _pool8(case, total, behind, gd):
    """The same in 8 bits: [pages, kv heads, 32 hd + 32] bytes, rows that were never written all ones."""
    nkv, hd = case["nkv"], case["hd"]
    pool = torch.empty((total, nkv, 32 * hd + 32), dtype=torch.uint8, device="cuda")
    size = torch.ones(hd, device="cuda")
    size[3::32] = 12.0  # a few channels of the keys are far larger than the others
    for side, off in enumerate(_offsets(hd, 1)):
        place = torch.empty(PAGE * hd, dtype=torch.int64)
        place[off.reshape(-1)] = torch.arange(PAGE * hd)
        place = place.cuda()
        for p in range(0, total, 4096):  # (a few pages at a time: the values of a long cache in 32 bits are large)
            n = min(4096, total - p)
            x = torch.randn((n, nkv, PAGE, hd), generator=gd, device="cuda")
            codes, exps = _quantised(x * size if side == 0 else x)
            codes[behind[p:p + n][:, None].expand(n, nkv, PAGE)] = 255
            pool[p:p + n, :, side * PAGE * hd:(side + 1) * PAGE * hd] = codes.view(n, nkv, -1)[:, :, place]
            pool[p:p + n, :, 32 * hd + side * PAGE:32 * hd + (side + 1) * PAGE] = exps.masked_fill(behind[p:p + n][:, None], 255)
    return pool


def prepare(case, seed):
    g = torch.Generator().manual_seed(seed)
    gd = torch.Generator(device="cuda").manual_seed(seed)
    op, dev, dt = case["op"], "cuda", _dtype(case)
    if op == "rotate":
        rows, nh, nkv, hd = case["rows"], case["nh"], case["nkv"], case["hd"]
        # queries and keys as a fused projection leaves them: slices of wider rows
        y = torch.randn((rows, (nh + 2 * nkv) * hd), generator=gd, device=dev).to(dt)
        inv, scale = _inv_freq(case)
        st = dict(case=case, q=y[:, :nh * hd].view(rows, nh, hd), k=y[:, nh * hd:(nh + nkv) * hd].view(rows, nkv, hd),
                  positions=torch.randint(0, case["far"], (rows,), generator=gd, device=dev).to(torch.int32),
                  inv_freq=inv.cuda(), scale=scale, q_out=torch.zeros((rows, nh, hd), dtype=dt, device=dev),
                  k_out=torch.zeros((rows, nkv, hd), dtype=dt, device=dev))
        return st
    ctx, new, total, table = _pages(case, g)
    T, nkv, hd = sum(new), case["nkv"], case["hd"]
    behind = _behind(ctx, new, table, total)
    st = dict(case=case, page_tables=table.cuda(), row_starts=_i32(_starts(new)), kv_lens=_i32([c + n for c, n in zip(ctx, new)]),
              max_new=max(new))
    if op == "keep":
        # the branch from a root to one of the last nodes, of every tree
        paths = []
        for par in _parents(new, seed):
            at, path = len(par) - 1, []
            while at >= 0:
                path.append(at)
                at = par[at]
            paths.append(path[::-1])
        longest = max(len(p) for p in paths) + 1
        st.update(pool=_pool16(case, total, behind, gd), ctx_lens=_i32(ctx), path_lens=_i32([len(p) for p in paths]),
                  path=_i32([p + [-1] * (longest - len(p)) for p in paths]))
        return st
    if op == "store8":
        seq = torch.repeat_interleave(torch.arange(case["nb"]), torch.tensor(new))
        idx = torch.cat([torch.arange(c, c + n) for c, n in zip(ctx, new)])
        slots = (table[seq, idx // PAGE].long() * PAGE + idx % PAGE).to(torch.int32)
        y = torch.randn((T, 4 * nkv * hd), generator=gd, device=dev)
        y[:, 3::32] *= 12.0
        y = y.to(dt)
        st.update(k=y[:, 2 * nkv * hd:3 * nkv * hd].view(T, nkv, hd), v=y[:, 3 * nkv * hd:].view(T, nkv, hd), slots=slots.cuda(),
                  pool=torch.zeros((total, nkv, 32 * hd + 32), dtype=torch.uint8, device=dev))
        return st
    nh = case["nh"]
    st.update(q=(torch.randn((T, nh, hd), generator=gd, device=dev) * (1.5 if op == "tree" else 0.9)).to(dt),
              pool=_pool16(case, total, behind, gd) if op == "tree" else _pool8(case, total, behind, gd),
              out=torch.zeros((T, nh, hd), dtype=dt, device=dev), lse=torch.zeros((T, nh), device=dev))
    if op == "tree" or case["tree"]:
        st["parents"] = _i32([p for par in _parents(new, seed) for p in par])
        words = _up(max(new), 64)
        st.update(max_nodes=max(new), positions=torch.zeros(T, dtype=torch.int32, device=dev),
                  masks=torch.zeros((T, words), dtype=torch.int64, device=dev))
    return st


# ------------------------------------------------------------------------------------- plain forms
def _rotate_plain(s):
    case = s["case"]
    r = case["rd"]
    angle = s["positions"].double()[:, None] * s["inv_freq"][None]
    c, n = (torch.cos(angle) * s["scale"]).float()[:, None], (torch.sin(angle) * s["scale"]).float()[:, None]
    for x, out in ((s["q"], s["q_out"]), (s["k"], s["k_out"])):
        x = x.float()
        if case["interleaved"]:
            a, b = x[..., 0:r:2], x[..., 1:r:2]
            y = torch.stack([a * c - b * n, b * c + a * n], -1).flatten(-2)
        else:
            a, b = x[..., :r // 2], x[..., r // 2:r]
            y = torch.cat([a * c - b * n, b * c + a * n], -1)
        out[..., :r] = y.to(out.dtype)
        out[..., r:] = x[..., r:].to(out.dtype)
    return s["q_out"], s["k_out"]


def _tree_plain(s):
    """positions [rows], masks [rows, words] and the trees' ancestors [nb, m, m]."""
    st, kv, par, m = s["row_starts"].long(), s["kv_lens"].long(), s["parents"].long(), s["max_new"]
    new = st[1:] - st[:-1]
    i = torch.arange(m, device=par.device)
    row = (st[:-1, None] + i[None]).clamp(max=par.numel() - 1)
    live = i[None] < new[:, None]
    p = torch.where(live, par[row], -1)
    reach = (p[:, :, None] == i[None, None]) & live[:, :, None] | torch.eye(m, dtype=torch.bool, device=par.device)
    hop = 1
    while hop < m:  # paths of twice the length
        reach = (reach.float() @ reach.float()) > 0
        hop *= 2
    reach &= live[:, :, None] & live[:, None, :]
    s["positions"][:] = ((kv - new)[:, None] + reach.sum(2) - 1)[live].to(torch.int32)
    words = s["masks"].shape[1]
    bits = torch.zeros((*reach.shape[:2], words * 64), dtype=torch.int64, device=par.device)
    bits[:, :, :m] = reach
    shifted = bits.view(*reach.shape[:2], words, 64) << torch.arange(64, device=par.device)
    s["masks"][:] = shifted.sum(-1)[live]
    return reach


def _rows16(pool, table):
    """K and V [nb, nkv, rows, hd] of the tables' pages in 32 bits."""
    nb, mpps = table.shape
    nkv, hd = pool.shape[1], pool.shape[3] // PAGE
    pg = pool[table]
    keys = pg[:, :, :, 0].view(nb, mpps, nkv, 2, hd // 8, 8, 8).permute(0, 2, 1, 3, 5, 4, 6).reshape(nb, nkv, -1, hd).float()
    return keys, pg[:, :, :, 1].view(nb, mpps, nkv, hd // 8, 2, 8, 8).permute(0, 2, 1, 4, 6, 3, 5).reshape(nb, nkv, -1, hd).float()


def _rows8(pool, table):
    nb, mpps = table.shape
    nkv, hd = pool.shape[1], (pool.shape[2] - 32) // 32
    pg = pool[table]
    got = []
    for side, off in enumerate(_offsets(hd, 1)):
        codes = pg[..., side * PAGE * hd:(side + 1) * PAGE * hd][..., off.reshape(-1).to(pg.device)].view(torch.float8_e4m3fn).float()
        exps = pg[..., 32 * hd + side * PAGE:32 * hd + (side + 1) * PAGE].to(torch.int32) - 127
        x = codes.view(nb, mpps, nkv, PAGE, hd) * _pow2(exps)[..., None]
        got.append(x.permute(0, 2, 1, 3, 4).reshape(nb, nkv, -1, hd))
    return got


def _attend_plain(s):
    case, q, table = s["case"], s["q"], s["page_tables"].long().clamp(min=0)
    T, nh, hd = q.shape
    nb, nkv, m = case["nb"], case["nkv"], s["max_new"]
    gq = nh // nkv
    kv, st = s["kv_lens"].long(), s["row_starts"].long()
    new = st[1:] - st[:-1]
    reach = _tree_plain(s) if "parents" in s else None
    # the sequences' rows, gathered from their pages and padded to one length
    keys, vals = _rows16(s["pool"], table) if case["op"] == "tree" else _rows8(s["pool"], table)
    j = torch.arange(keys.shape[2], device=q.device)
    live = (j[None] < kv[:, None])[:, None, :, None]
    keys, vals = torch.where(live, keys, 0.0), torch.where(live, vals, 0.0)
    # the queries, padded to [nb, m]
    i = torch.arange(m, device=q.device)
    row = (st[:-1, None] + i[None]).clamp(max=T - 1)
    qp = q[row].float().view(nb, m, nkv, gq, hd).permute(0, 2, 3, 1, 4).reshape(nb, nkv, gq * m, hd)
    sc = qp @ keys.transpose(2, 3) * (1.0 / math.sqrt(hd))
    ctx = kv - new
    if reach is None:
        pos = ctx[:, None] + i[None]
        see = (j[None, None] <= pos[:, :, None]) & (j[None, None] < kv[:, None, None])
        far = pos[:, :, None] - j[None, None]
    else:
        pos = ctx[:, None] + reach.sum(2) - 1
        own_row = j[None] - ctx[:, None]
        at = own_row.clamp(0, m - 1)[:, None].expand(nb, m, -1)
        see = torch.where((own_row < 0)[:, None], True, reach.gather(2, at) & (own_row < new[:, None])[:, None])
        far = torch.where((own_row < 0)[:, None], pos[:, :, None] - j[None, None], 0)
    if case["window"] > 0:
        see &= far < case["window"]
    sc = sc.view(nb, nkv, gq, m, -1).masked_fill_(~see[:, None, None], float("-inf"))
    top = sc.amax(-1, keepdim=True)
    top = torch.where(top == float("-inf"), 0.0, top)
    sc = sc.sub_(top).exp_()
    total = sc.sum(-1, keepdim=True)
    o = (sc.view(nb, nkv, gq * m, -1) @ vals).view(nb, nkv, gq, m, hd) / torch.where(total > 0, total, 1.0)
    lse = torch.log(total) + top
    take = i[None] < new[:, None]
    s["out"][:] = o.permute(0, 3, 1, 2, 4).reshape(nb, m, nh, hd)[take].to(q.dtype)
    s["lse"][:] = lse[..., 0].permute(0, 3, 1, 2).reshape(nb, m, nh)[take]
    return (s["positions"], s["masks"], s["out"], s["lse"]) if "parents" in s else (s["out"], s["lse"])


def _keep_plain(s):
    pool, table, path = s["pool"], s["page_tables"].long(), s["path"].long()
    nkv, hd = pool.shape[1], pool.shape[3] // PAGE
    i = torch.arange(path.shape[1], device=pool.device)
    live = i[None] < s["path_lens"].long()[:, None]
    seq, step = live.nonzero(as_tuple=True)
    src, dst = (s["ctx_lens"].long()[seq] + path[seq, step]), (s["ctx_lens"].long()[seq] + step)
    h = torch.arange(nkv, device=pool.device)[None, :, None]
    flat = pool.view(-1)
    places = []
    for at in (src, dst):
        page, j = table[seq, at // PAGE], at % PAGE
        tile = (page[:, None, None] * nkv + h) * (2 * PAGE * hd)
        ko, vo = (o.to(pool.device)[j][:, None] for o in _offsets(hd, 2))
        places.append(torch.cat([tile + ko, tile + PAGE * hd + vo], -1))
    flat[places[1]] = flat[places[0]]
    return pool


def _store8_plain(s):
    pool, slots, dt = s["pool"], s["slots"].long(), s["k"].dtype
    nkv, hd = s["k"].shape[1:]
    page, j = slots // PAGE, slots % PAGE
    h = torch.arange(nkv, device=pool.device)[None, :]
    got = []
    for side, x in ((0, s["k"]), (1, s["v"])):
        codes, exps = _quantised(x)
        at = _offsets(hd, 1)[side].to(pool.device)[j][:, None] + side * PAGE * hd
        pool[page[:, None, None], h[..., None], at] = codes
        pool[page[:, None], h, (32 * hd + side * PAGE + j)[:, None]] = exps
        back = pool[page[:, None, None], h[..., None], at].view(torch.float8_e4m3fn).float()
        k = pool[page[:, None], h, (32 * hd + side * PAGE + j)[:, None]].to(torch.int32) - 127
        got.append((back * _pow2(k)[..., None]).to(dt))
    return tuple(got)


def run(state):
    s, op = state, state["case"]["op"]
    if own:
        from block_diffusion_drafter_forward_gb300 import PagedKV, QuantKV, Rope, TreePlan, draft_tree
        if op == "rotate":
            case = s["case"]
            kind = case["rd"], case["theta"], case["scaling"], case["interleaved"]
            if kind not in _ropes:  # a table of frequencies that a user's program makes once
                _ropes[kind] = Rope(case["rd"], theta=case["theta"], linear=4.0 if case["scaling"] == "linear" else 1.0,
                                    yarn=_yarn(case), interleaved=case["interleaved"])
            return _ropes[kind].rotate(s["q"], s["positions"], k=s["k"], out=s["q_out"], k_out=s["k_out"])
        if op == "keep":
            return PagedKV(s["pool"]).keep(s["page_tables"], s["ctx_lens"], s["path"], s["path_lens"])
        if op == "store8":
            kv = QuantKV(s["pool"])
            kv.append(s["k"], s["v"], s["slots"])
            return kv.read(s["slots"], dtype=s["k"].dtype)
        kv, tree = (PagedKV if op == "tree" else QuantKV)(s["pool"]), None
        if "parents" in s:
            tree = draft_tree(s["parents"], s["kv_lens"], s["row_starts"], s["max_nodes"], out=TreePlan(s["positions"], s["masks"]))
        got = kv.attend(s["q"], s["page_tables"], s["kv_lens"], s["row_starts"], s["max_new"], window=s["case"]["window"],
                        tree=tree, out=s["out"], lse=s["lse"])
        return (s["positions"], s["masks"]) + got if tree is not None else got
    return {"rotate": _rotate_plain, "keep": _keep_plain, "store8": _store8_plain, "tree": _attend_plain, "attend8": _attend_plain}[op](s)


# ------------------------------------------------------------------------------------- work
def work(case):
    op, es = case["op"], 4 if case.get("dtype") == "f32" else 2
    if op == "rotate":
        n = case["rows"] * (case["nh"] + case["nkv"])
        return {"bytes": 2 * n * case["hd"] * es + 4 * case["rows"], "flops": 3 * n * case["rd"]}
    ctx, new = _lens(case)
    nb, T, nkv, hd = case["nb"], sum(new), case["nkv"], case["hd"]
    if op == "keep":  # about a third of a tree's nodes lie on a branch
        n = sum(_up(x, 3) for x in new)
        return {"bytes": 2 * n * 2 * nkv * hd * es + 4 * n + 8 * nb, "flops": 0}
    if op == "store8":  # rows in, codes out and in, rows out
        return {"bytes": T * 2 * nkv * (2 * hd * es + 2 * (hd + 1)) + 8 * T, "flops": 4 * T * nkv * hd}
    nh, W = case["nh"], case["window"]
    tree = op == "tree" or case["tree"]
    pairs = rows = 0
    for c, n in zip(ctx, new):
        if n:
            rows += c + n - (max(0, c + 1 - W) if W > 0 else 0)
            seen = n * (min(c, W) if W > 0 else c) + n * 8 if tree else n * c + n * (n + 1) // 2
            if W > 0 and not tree:  # row at position p loses max(0, p + 1 - W) keys
                a, b = max(c + 1, W + 1), c + n
                if b >= a:
                    seen -= (b - a + 1) * (a - W + b - W) // 2
            pairs += seen
    per_row = 2 * hd * 2 if op == "tree" else 2 * (hd + 1)
    extra = T * (4 + 4 + 8 * _up(max(new), 64)) if tree else 0
    return {"bytes": rows * nkv * per_row + 2 * (2 * T * nh * hd) + 4 * T * nh + extra, "flops": 4 * hd * nh * pairs}


# ------------------------------------------------------------------------------------- 64 bits
def _unit(k):
    """2^k in 64 bits."""
    return ((k.to(torch.int64) + 1023) << 52).view(torch.float64)


def _e4m3(y):
    """The nearest e4m3 value of |y| <= 448 (ties to even), in 64 bits."""
    _, e = torch.frexp(y)
    step = _unit((e - 1).clamp(min=-6) - 3)
    return torch.round(y / step) * step


def _decoded(byte):
    """e4m3 codes as numbers, by sign, exponent and mantissa."""
    b = byte.to(torch.int64)
    e, m = b >> 3 & 15, (b & 7).double()
    v = torch.where(e > 0, (1 + m / 8) * _unit(e - 7), m / 8 * 2.0 ** -6)
    return torch.where(b >= 128, -v, v)


def exact(case, seed):
    op = case["op"]
    s = prepare(case, seed)
    if op == "rotate":
        inv, scale = _inv_freq(case)
        r, turn = case["rd"], s["positions"].double()[:, None] * inv.cuda()[None]
        unit = torch.polar(torch.full_like(turn, scale), turn)[:, None]
        got = []
        for x in (s["q"].double(), s["k"].double()):
            y = x.clone()
            if case["interleaved"]:
                z = torch.view_as_complex(x[..., :r].reshape(*x.shape[:2], r // 2, 2).contiguous()) * unit
                y[..., :r] = torch.view_as_real(z).reshape(*x.shape[:2], r)
            else:
                z = torch.complex(x[..., :r // 2].contiguous(), x[..., r // 2:r].contiguous()) * unit
                y[..., :r // 2], y[..., r // 2:r] = z.real, z.imag
            got.append(y)
        return tuple(got)
    ctx, new = _lens(case)
    nkv, hd, nb = case["nkv"], case["hd"], case["nb"]
    if op == "store8":
        got = []
        for x in (s["k"].double(), s["v"].double()):
            top = x.abs().amax(-1, keepdim=True)
            k = torch.full_like(top, -118.0)
            lg = torch.ceil(torch.log2(top.clamp(min=1e-300) / 448.0))
            for c in (lg - 1, lg, lg + 1):  # (a logarithm next to a whole number may be off: the definition decides)
                k = torch.where((k == -118.0) & (top <= 448.0 * _unit(c.clamp(-1000, 1000))) & (top > 0), c.clamp(-118, 119), k)
            unit = _unit(k)
            got.append(_e4m3((x / unit).clamp(-448.0, 448.0)) * unit)
        return tuple(got)
    table = s["page_tables"]
    if op == "keep":
        pool = s["pool"].double()
        ko, vo = (o.to(pool.device) for o in _offsets(hd, 2))
        old = pool.clone()
        for b in range(nb):
            for i, p in enumerate(s["path"][b, :int(s["path_lens"][b])].tolist()):
                a, z = ctx[b] + p, ctx[b] + i
                pa, pz = int(table[b, a // PAGE]), int(table[b, z // PAGE])
                pool[pz, :, 0, ko[z % PAGE]] = old[pa, :, 0, ko[a % PAGE]]
                pool[pz, :, 1, vo[z % PAGE]] = old[pa, :, 1, vo[a % PAGE]]
        return pool
    q, pool, nh = s["q"], s["pool"], case["nh"]
    if 4 * hd * nh * sum(n * (c + n) for c, n in zip(ctx, new)) > 6e12:
        return None
    tree = "parents" in s
    trees = _parents(new, seed)
    out = torch.zeros(q.shape, dtype=torch.float64, device="cuda")
    lse = torch.zeros(q.shape[:2], dtype=torch.float64, device="cuda")
    ko, vo = (o.to(pool.device) for o in _offsets(hd, 2 if op == "tree" else 1))
    at = 0
    for b, (c, n) in enumerate(zip(ctx, new)):
        if not n:
            continue
        L = c + n
        key = torch.arange(L, device="cuda")
        page, j = table[b, key // PAGE].long(), key % PAGE
        far = (c + torch.arange(n, device="cuda"))[:, None] - key[None]
        hide = far < 0
        if tree:
            see, depth = [[False] * n for _ in range(n)], []
            for i, p in enumerate(trees[b]):
                if p >= 0:
                    see[i] = list(see[p])
                see[i][i] = True
                depth.append(depth[p] + 1 if p >= 0 else 0)
            hide[:, c:] = ~torch.tensor(see, device="cuda")
            far = (c + torch.tensor(depth, device="cuda"))[:, None] - key[None]
            far[:, c:] = 0
        if case["window"] > 0:
            hide = hide | (far >= case["window"])
        for g in range(nkv):
            if op == "tree":
                tile = (page * nkv + g)[:, None] * (2 * PAGE * hd)
                K, V = pool.view(-1)[tile + ko[j]].double(), pool.view(-1)[tile + PAGE * hd + vo[j]].double()
            else:
                tile = (page * nkv + g)[:, None] * (32 * hd + 32)
                flat = pool.view(-1)
                K = _decoded(flat[tile + ko[j]]) * _unit(flat[tile + 32 * hd + j[:, None]].int() - 127)
                V = _decoded(flat[tile + PAGE * hd + vo[j]]) * _unit(flat[tile + 32 * hd + PAGE + j[:, None]].int() - 127)
            for h in range(g * (nh // nkv), (g + 1) * (nh // nkv)):
                z = (q[at:at + n, h].double() @ K.t() / math.sqrt(hd)).masked_fill(hide, float("-inf"))
                l = torch.logsumexp(z, 1)
                lse[at:at + n, h] = l
                out[at:at + n, h] = torch.exp(z - l[:, None]) @ V
        at += n
    return (None, None, out, lse) if tree else (out, lse)
