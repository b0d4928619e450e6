"""Cases of the serving operators around the drafter: what a target model's step over a paged K/V
cache calls before and after its projections.

  tables   extend_tables: new rows of a batch get their pages, row map and slots on the device
  append   PagedKV.append: K and V rows of the step scattered into the pages by slot
  attend   PagedKV.attend: a chunk of new tokens per sequence (one token, a block to verify, a
           prompt) attends over its paged rows, causal, with an optional window
  sample   sample: one token per logits row from a given uniform number, by temperature, top-k,
           top-p and min-p

`run` computes an operator in plain torch operations, or (own = True) through the package's entry
points.  Lengths are a function of the case alone; values, page ids and random numbers of the seed.
"""
import math
import random

import torch

own = False
PAGE = 16


# ------------------------------------------------------------------------------------- cases
def listed():
    return [
        # one verification step of a batch: every sequence gets a block of 16 rows
        dict(name="tables_verify_64x16", op="tables", nb=64, new_lo=16, new_hi=16, ctx_lo=512, ctx_hi=8192),
        # prompts of very different lengths admitted together (ragged, some sequences add nothing)
        dict(name="tables_prompts_512", op="tables", nb=512, new_lo=0, new_hi=511, ctx_lo=0, ctx_hi=16384),
        # K/V of that verification step: 64 sequences x 16 rows, the 8-layer drafter's K/V heads
        dict(name="append_verify_64x16", op="append", nb=64, new_lo=16, new_hi=16, ctx_lo=512, ctx_hi=8192,
             nkv=4, hd=128, dtype="bf16"),
        # K/V of a prefill step: ragged prompts of 16 Ki rows together, 8 K/V heads
        dict(name="append_prompts_24", op="append", nb=24, new_lo=33, new_hi=1333, ctx_lo=0, ctx_hi=700,
             nkv=8, hd=128, dtype="bf16"),
        # one sequence decoding one token at the benchmark's context: latency
        dict(name="attend_decode_1x4096", op="attend", nb=1, new_lo=1, new_hi=1, ctx_lo=4096, ctx_hi=4096,
             nh=32, nkv=4, hd=128, window=0),
        # the benchmark's ragged batch, every sequence verifying a block of 16 tokens
        dict(name="attend_verify_32x16", op="attend", nb=32, new_lo=16, new_hi=16, ctx_lo=512, ctx_hi=8192,
             nh=32, nkv=4, hd=128, window=0),
        # long-context decoding, the wide drafter's heads
        dict(name="attend_decode_16x32768", op="attend", nb=16, new_lo=1, new_hi=1, ctx_lo=16001, ctx_hi=32767,
             nh=64, nkv=8, hd=128, window=0),
        # one long prompt in one chunk
        dict(name="attend_prompt_8192", op="attend", nb=1, new_lo=8192, new_hi=8192, ctx_lo=0, ctx_hi=0,
             nh=32, nkv=4, hd=128, window=0),
        # a mixed step: prompts' chunks and single tokens together, on the wide drafter's sliding layers
        dict(name="attend_mixed_8_window", op="attend", nb=8, new_lo=0, new_hi=777, ctx_lo=0, ctx_hi=3001,
             nh=64, nkv=8, hd=128, window=2048),
        # one sequence drawing its next token
        dict(name="sample_1", op="sample", rows=1, vocab=151936, dtype="bf16", preset="nucleus"),
        # a decode step of 64 sequences with settings of their own, fp32 logits, the largest vocabulary
        dict(name="sample_64_f32", op="sample", rows=64, vocab=262144, dtype="f32", preset="mixed"),
        # every row of a verification step: 64 sequences x 16 rows
        dict(name="sample_1024", op="sample", rows=1024, vocab=151936, dtype="bf16", preset="mixed"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("tables", "append", "attend", "attend", "sample"))
    if op == "tables":
        lo = rng.choice((0, 1))
        return dict(op=op, nb=_log(rng, 1, 512), new_lo=lo, new_hi=lo + _log(rng, 1, 511), ctx_lo=0,
                    ctx_hi=_log(rng, 16, 16384))
    if op == "append":
        hd = rng.choice((64, 128))
        nb = _log(rng, 1, 64)
        lo = rng.choice((0, 1))
        return dict(op=op, nb=nb, new_lo=lo, new_hi=lo + _log(rng, 1, max(1, 16384 // nb)), ctx_lo=0,
                    ctx_hi=_log(rng, 16, 1000), nkv=rng.choice((1, 2, 4, 8)), hd=hd, dtype=rng.choice(("bf16", "f32")))
    if op == "attend":
        nkv, group, hd = rng.choice((1, 2, 4, 8)), rng.choice((1, 4, 5, 8, 16)), rng.choice((64, 128))
        group = min(group, 64 // nkv)
        window = rng.choice((0, 0, _log(rng, 100, 2048)))
        form = rng.choice(("single", "block", "prompt"))
        if form == "single":
            nb = _log(rng, 1, 64)
            hi = _log(rng, 64, min(32768, 262144 // nb))
            return dict(op=op, nb=nb, new_lo=1, new_hi=1, ctx_lo=hi // 2, ctx_hi=hi, nh=nkv * group, nkv=nkv, hd=hd,
                        window=window)
        if form == "block":
            nb = _log(rng, 1, 32)
            hi = _log(rng, 64, 8192)
            return dict(op=op, nb=nb, new_lo=1, new_hi=rng.randint(2, 16), ctx_lo=hi // 4, ctx_hi=hi, nh=nkv * group,
                        nkv=nkv, hd=hd, window=window)
        nb = rng.randint(1, 6)
        return dict(op=op, nb=nb, new_lo=0, new_hi=_log(rng, 17, 1500), ctx_lo=0, ctx_hi=_log(rng, 16, 2500),
                    nh=nkv * group, nkv=nkv, hd=hd, window=window)
    vocab = rng.choice((2048, 8192, 151936, 262144, rng.randint(1000, 200000)))
    return dict(op=op, rows=_log(rng, 1, max(1, 64 * 1024 * 1024 // vocab)), vocab=vocab,
                dtype=rng.choice(("bf16", "f32")), preset=rng.choice(("mixed", "nucleus", "plain", "top_k")))


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


# ------------------------------------------------------------------------------------- inputs
def _cache(case, seed, g):
    """Page tables of a shared pool: each sequence's pages are a run of one random permutation."""
    ctx, new = _lens(case)
    pages = [_up(c + n, PAGE) for c, n in zip(ctx, new)]
    mpps = max(max(pages), 1) + 2
    total = sum(pages) + 3
    perm = torch.randperm(total, generator=g).to(torch.int32)
    return ctx, new, pages, mpps, total, perm


def _table(pages, mpps, perm):
    t = torch.full((len(pages), mpps), -1, dtype=torch.int32)
    at = 0
    for s, n in enumerate(pages):
        t[s, :n] = perm[at:at + n]
        at += n
    return t


def _i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _starts(new):
    out = [0]
    for n in new:
        out.append(out[-1] + n)
    return out


def _settings(preset, rows, r):
    """(temperature, top_k, top_p, min_p) of every row, as serving requests carry them."""
    sets = {"nucleus": [(0.7, 0, 0.95, 0.0)], "plain": [(1.0, 0, 1.0, 0.0), (0.8, 0, 1.0, 0.0)],
            "top_k": [(0.6, 20, 0.95, 0.0), (1.0, 50, 1.0, 0.0)],
            "mixed": [(0.0, 0, 1.0, 0.0), (1.0, 0, 1.0, 0.0), (0.7, 50, 0.95, 0.0), (0.8, 0, 0.95, 0.0),
                      (1.2, 0, 1.0, 0.05), (0.6, 20, 0.95, 0.0), (0.9, 1000, 0.8, 0.02)]}[preset]
    return [sets[(i + r) % len(sets)] for i in range(rows)]


def prepare(case, seed):
    g = torch.Generator().manual_seed(seed)
    gd = torch.Generator(device="cuda").manual_seed(seed)
    op = case["op"]
    dev = "cuda"
    if op == "sample":
        rows, V = case["rows"], case["vocab"]
        dt = torch.bfloat16 if case["dtype"] == "bf16" else torch.float32
        # a language model's row: a broad body and a few dozen likely tokens with falling scores
        x = torch.randn((rows, V), generator=gd, device=dev) * 2.0
        # (one place in each of 48 equal parts of the vocabulary: no place twice, so that a write has one value)
        top = torch.rand((rows, 48), generator=gd, device=dev).argsort(1) * (V // 48) + torch.randint(V // 48, (rows, 48), generator=gd, device=dev)
        rank = torch.arange(48, device=dev, dtype=torch.float32)
        x.scatter_(1, top, 17.0 - 1.7 * torch.log1p(rank) + torch.randn((rows, 48), generator=gd, device=dev))
        st = _settings(case["preset"], rows, seed % 7)
        cols = list(zip(*st))
        return dict(case=case, logits=x.to(dt), u=torch.rand(rows, generator=gd, device=dev),
                    temperature=torch.tensor(cols[0], device=dev), top_k=_i32(cols[1]),
                    top_p=torch.tensor(cols[2], device=dev), min_p=torch.tensor(cols[3], device=dev),
                    tokens=torch.empty(rows, dtype=torch.int32, device=dev),
                    probs=torch.empty(rows, dtype=torch.float32, device=dev))
    ctx, new, pages, mpps, total, perm = _cache(case, seed, g)
    starts, T = _starts(new), sum(new)
    st = dict(case=case, row_starts=_i32(starts))
    if op == "tables":
        held = [_up(c, PAGE) for c in ctx]
        table = torch.full((case["nb"], mpps), -1, dtype=torch.int32)
        at = 0
        for s, n in enumerate(held):
            table[s, :n] = perm[at:at + n]
            at += n
        free = torch.cat([perm[:2], perm[at:]])  # a stack of free pages whose first two are taken already
        rows = T + 5                             # room for a few rows more than the step has
        i32 = dict(dtype=torch.int32, device=dev)
        st.update(ctx_lens=_i32(ctx), new_rows=_i32(new), page_tables=table.cuda(), free_pages=free.cuda(),
                  free_begin=_i32([2]), max_rows=rows,
                  out=(torch.empty(case["nb"], **i32), torch.empty(case["nb"] + 1, **i32), torch.empty(rows, **i32),
                       torch.empty(rows, **i32), torch.empty(rows, **i32), torch.empty(1, **i32)))
        return st
    nkv, hd = case["nkv"], case["hd"]
    table = _table(pages, mpps, perm)
    # slots of the step's rows, from the tables
    seq = torch.repeat_interleave(torch.arange(case["nb"]), torch.tensor(new))
    idx = torch.cat([torch.arange(c, c + n) for c, n in zip(ctx, new)])
    slots = (table[seq, idx // PAGE].long() * PAGE + idx % PAGE).to(torch.int32)
    if op == "append":
        dt = torch.bfloat16 if case["dtype"] == "bf16" else torch.float32
        # K and V rows as a fused projection leaves them: slices of wider rows
        y = torch.randn((T, 4 * nkv * hd), generator=gd, device=dev).to(dt)
        st.update(k=y[:, 2 * nkv * hd:3 * nkv * hd].view(T, nkv, hd), v=y[:, 3 * nkv * hd:].view(T, nkv, hd),
                  slots=slots.cuda(), pool=torch.zeros((total, nkv, 2, PAGE * hd), dtype=dt, device=dev))
        return st
    bf = torch.bfloat16
    # rows of the pages hold unit keys and values; rows past a sequence's end were never written: NaN
    pool = torch.randn((total, nkv, 2, PAGE * hd), generator=gd, device=dev).to(bf)
    for s, (c, n) in enumerate(zip(ctx, new)):
        if (c + n) % PAGE:
            p, j = int(table[s, (c + n) // PAGE]), (c + n) % PAGE
            off = torch.arange(j, PAGE)
            kk = ((off[:, None] // 8) * (hd // 8) + torch.arange(hd)[None] // 8) * 64 + (off[:, None] % 8) * 8 + torch.arange(hd)[None] % 8
            vv = ((torch.arange(hd)[None] // 8) * 2 + off[:, None] // 8) * 64 + (torch.arange(hd)[None] % 8) * 8 + off[:, None] % 8
            pool[p, :, 0, kk.reshape(-1).cuda()] = float("nan")
            pool[p, :, 1, vv.reshape(-1).cuda()] = float("nan")
    nh = case["nh"]
    # queries of a trained model are larger than unit: scores spread over a few units
    q = (torch.randn((T, nh, hd), generator=gd, device=dev) * 1.5).to(bf)
    st.update(q=q, pool=pool, page_tables=table.cuda(), kv_lens=_i32([c + n for c, n in zip(ctx, new)]), max_new=max(new),
              out=torch.zeros((T, nh, hd), dtype=bf, device=dev), lse=torch.zeros((T, nh), device=dev))
    return st


# ------------------------------------------------------------------------------------- plain forms
def _tables_plain(s):
    ctx, n, table = s["ctx_lens"].long(), s["new_rows"].long(), s["page_tables"]
    nb, mpps = table.shape
    rows, free = s["max_rows"], s["free_pages"]
    valid = (ctx >= 0) & (n >= 0) & (ctx + n <= mpps * PAGE)
    held = (ctx + PAGE - 1) // PAGE
    need = torch.where(valid, (ctx + n + PAGE - 1) // PAGE - held, 0)
    n = torch.where(valid, n, 0)
    pages_to, rows_to = torch.cumsum(need, 0), torch.cumsum(n, 0)
    begin = s["free_begin"].long()
    fits = (begin + pages_to <= free.numel()) & (rows_to <= rows)
    need, n = torch.where(fits, need, 0), torch.where(fits, n, 0)
    pages_to, rows_to = torch.cumsum(need, 0), torch.cumsum(n, 0)
    i = torch.arange(free.numel(), device=table.device)
    at = torch.searchsorted(pages_to, i, right=True)
    live = at < nb
    at, i = at[live], i[live]
    table[at, held[at] + i - (pages_to - need)[at]] = free[begin + i]
    r = torch.arange(rows, device=table.device)
    seq = torch.searchsorted(rows_to, r, right=True)
    live = seq < nb
    sq = torch.where(live, seq, 0)
    idx = ctx[sq] + r - (rows_to - n)[sq]
    idx_in = torch.where(live, idx, 0)
    slot = table[sq, idx_in // PAGE].long() * PAGE + idx_in % PAGE
    i32 = torch.int32
    return (table, (ctx + n).to(i32), torch.cat([torch.zeros_like(rows_to[:1]), rows_to]).to(i32),
            torch.where(live, seq, -1).to(i32), torch.where(live, idx, -1).to(i32), torch.where(live, slot, -1).to(i32),
            (begin + pages_to[-1:]).to(i32))


def _append_plain(s):
    k, v, pool, slots = s["k"], s["v"], s["pool"], s["slots"].long()
    n, nkv, hd = k.shape
    P = pool.shape[0]
    ok = slots >= 0
    page, j = slots[ok] // PAGE, slots[ok] % PAGE
    kt = pool[:, :, 0].view(P, nkv, 2, hd // 8, 8, 8)
    vt = pool[:, :, 1].view(P, nkv, hd // 8, 2, 8, 8)
    kt[page, :, j // 8, :, j % 8, :] = k[ok].reshape(-1, nkv, hd // 8, 8)
    vt[page, :, :, j // 8, :, j % 8] = v[ok].reshape(-1, nkv, hd // 8, 8)
    return pool


def _attend_plain(s):
    case, q, pool, table = s["case"], s["q"], s["pool"], s["page_tables"].long()
    T, nh, hd = q.shape
    nb, mpps = table.shape
    nkv = pool.shape[1]
    gq = nh // nkv
    kv, st = s["kv_lens"].long(), s["row_starts"].long()
    new = st[1:] - st[:-1]
    m = s["max_new"]
    # the sequences' rows, gathered from their pages and padded to one length
    pg = pool[table.clamp(min=0)]
    keys = pg[:, :, :, 0].view(nb, mpps, nkv, 2, hd // 8, 8, 8).permute(0, 2, 1, 3, 5, 4, 6).reshape(nb, nkv, -1, hd).float()
    vals = pg[:, :, :, 1].view(nb, mpps, nkv, hd // 8, 2, 8, 8).permute(0, 2, 1, 4, 6, 3, 5).reshape(nb, nkv, -1, hd).float()
    j = torch.arange(mpps * PAGE, device=q.device)
    live = (j[None] < kv[:, None])[:, None, :, None]
    keys, vals = torch.where(live, keys, 0.0), torch.where(live, vals, 0.0)
    # the queries, padded to [nb, m]
    i = torch.arange(m, device=q.device)
    row = (st[:-1, None] + i[None]).clamp(max=T - 1)
    qp = q[row].float().view(nb, m, nkv, gq, hd).permute(0, 2, 3, 1, 4).reshape(nb, nkv, gq * m, hd)
    sc = qp @ keys.transpose(2, 3) * (1.0 / math.sqrt(hd))
    pos = (kv - new)[:, None] + i[None]
    see = (j[None, None] <= pos[:, :, None]) & (j[None, None] < kv[:, None, None])
    if case["window"] > 0:
        see &= pos[:, :, None] - j[None, None] < case["window"]
    sc = sc.view(nb, nkv, gq, m, -1).masked_fill_(~see[:, None, None], float("-inf"))
    top = sc.amax(-1, keepdim=True)
    top = torch.where(top == float("-inf"), 0.0, top)
    sc = sc.sub_(top).exp_()
    total = sc.sum(-1, keepdim=True)
    o = (sc.view(nb, nkv, gq * m, -1) @ vals).view(nb, nkv, gq, m, hd) / torch.where(total > 0, total, 1.0)
    lse = torch.log(total) + top
    take = (i[None] < new[:, None])
    s["out"][:] = o.permute(0, 3, 1, 2, 4).reshape(nb, m, nh, hd)[take].to(q.dtype)
    s["lse"][:] = lse[..., 0].permute(0, 3, 1, 2).reshape(nb, m, nh)[take]
    return s["out"], s["lse"]


def _sample_plain(s):
    x = s["logits"].double()
    rows, V = x.shape
    T, p, lo, u = s["temperature"].double()[:, None], s["top_p"].double()[:, None], s["min_p"].double()[:, None], s["u"].double()
    k = s["top_k"].long()[:, None]
    xs, order = torch.sort(x, dim=1, descending=True, stable=True)
    T1 = torch.where(T > 0, T, 1.0)
    w = torch.exp((xs - xs[:, :1]) / T1)
    w = torch.where(w < 2.0 ** -40, 0.0, w)
    at = torch.arange(V, device=x.device)[None]
    keep = (at < torch.where(k > 0, k, V)) & torch.where(T > 0, True, at == 0)
    w = torch.where(keep, w, 0.0)
    before = torch.cumsum(w, 1) - w
    keep = ((p >= 1.0) | (before < p * w.sum(1, keepdim=True)) | (at == 0)) & (w >= lo)
    w = torch.where(keep, w, 0.0)
    by_index = torch.zeros_like(x).scatter_(1, order, w)
    run = torch.cumsum(by_index, 1)
    total = run[:, -1:]
    token = (run <= u[:, None] * total).sum(1, keepdim=True).clamp(max=V - 1)
    return token[:, 0].to(torch.int32), (by_index.gather(1, token) / total)[:, 0].float()


def run(state):
    op = state["case"]["op"]
    if own:
        from block_diffusion_drafter_forward_gb300 import PagedKV, RowPlan, extend_tables, sample
        s = state
        if op == "tables":
            r = extend_tables(s["ctx_lens"], s["new_rows"], s["page_tables"], s["free_pages"], s["free_begin"],
                              s["max_rows"], out=RowPlan(*s["out"]))
            return (s["page_tables"],) + tuple(r)
        if op == "append":
            return PagedKV(s["pool"]).append(s["k"], s["v"], s["slots"])
        if op == "attend":
            return PagedKV(s["pool"]).attend(s["q"], s["page_tables"], s["kv_lens"], s["row_starts"], s["max_new"],
                                             window=s["case"]["window"], out=s["out"], lse=s["lse"])
        return sample(s["logits"], s["u"], temperature=s["temperature"], top_k=s["top_k"], top_p=s["top_p"],
                      min_p=s["min_p"], tokens=s["tokens"], probs=s["probs"])
    return {"tables": _tables_plain, "append": _append_plain, "attend": _attend_plain, "sample": _sample_plain}[op](state)


# ------------------------------------------------------------------------------------- work
def work(case):
    if case["op"] == "sample":
        n = case["rows"] * case["vocab"]
        return {"bytes": n * (2 if case["dtype"] == "bf16" else 4) + 28 * case["rows"], "flops": 4 * n}
    ctx, new = _lens(case)
    nb, T = case["nb"], sum(new)
    if case["op"] == "tables":
        added = sum(_up(c + n, PAGE) - _up(c, PAGE) for c, n in zip(ctx, new))
        # lengths in, tables' new entries from the stack; per row: sequence, index, slot
        return {"bytes": 4 * (2 * nb + 2 * nb + 3 + 2 * added + 3 * (T + 5) + nb), "flops": 8 * T}
    nkv, hd = case["nkv"], case["hd"]
    if case["op"] == "append":
        es = 2 if case["dtype"] == "bf16" else 4
        return {"bytes": 4 * T * nkv * hd * es + 4 * T, "flops": 0}
    nh, W = case["nh"], case["window"]
    pairs = rows = 0
    for c, n in zip(ctx, new):
        if n:
            rows += c + n - (max(0, c + 1 - W) if W > 0 else 0)
            seen = n * c + n * (n + 1) // 2
            if W > 0:  # row at position p loses max(0, p + 1 - W) keys
                a, b = max(c + 1, W + 1), c + n
                if b >= a:
                    seen -= (b - a + 1) * (a - W + b - W) // 2
            pairs += seen
    return {"bytes": 2 * (rows * 2 * nkv * hd + 2 * T * nh * hd) + 4 * T * nh, "flops": 4 * hd * nh * pairs}


# ------------------------------------------------------------------------------------- 64 bits
def exact(case, seed):
    op = case["op"]
    if op == "tables":
        return None  # whole numbers only
    s = prepare(case, seed)
    if op == "append":
        k, v, pool, slots = s["k"].double(), s["v"].double(), s["pool"].double(), s["slots"].long()
        n, nkv, hd = k.shape
        flat = pool.view(-1)
        d, h = torch.arange(hd, device="cuda")[None, None], torch.arange(nkv, device="cuda")[None, :, None]
        page, j = (slots // PAGE)[:, None, None], (slots % PAGE)[:, None, None]
        tile = (page * nkv + h) * (2 * PAGE * hd)
        flat[tile + ((j // 8) * (hd // 8) + d // 8) * 64 + (j % 8) * 8 + d % 8] = k
        flat[tile + PAGE * hd + ((d // 8) * 2 + j // 8) * 64 + (d % 8) * 8 + j % 8] = v
        return pool
    if op == "attend":
        ctx, new = _lens(case)
        q, pool, table, nkv, hd, nh = s["q"], s["pool"], s["page_tables"], case["nkv"], case["hd"], case["nh"]
        if 4 * hd * nh * sum(n * (c + n) for c, n in zip(ctx, new)) > 6e12:
            return None
        out, lse, at = torch.zeros(q.shape, dtype=torch.float64, device="cuda"), torch.zeros(q.shape[:2], dtype=torch.float64, device="cuda"), 0
        d = torch.arange(hd, device="cuda")[None]
        for b, (c, n) in enumerate(zip(ctx, new)):
            L = c + n
            key = torch.arange(L, device="cuda")
            page, j = table[b, key // PAGE].long()[:, None], (key % PAGE)[:, None]
            for g in range(nkv if n else 0):
                tile = (page * nkv + g) * (2 * PAGE * hd)
                K = pool.view(-1)[tile + ((j // 8) * (hd // 8) + d // 8) * 64 + (j % 8) * 8 + d % 8].double()
                Vv = pool.view(-1)[tile + PAGE * hd + ((d // 8) * 2 + j // 8) * 64 + (d % 8) * 8 + j % 8].double()
                far = (c + torch.arange(n, device="cuda"))[:, None] - key[None]
                hide = far < 0
                if case["window"] > 0:
                    hide = hide | (far >= case["window"])
                for h in range(g * (nh // nkv), (g + 1) * (nh // nkv)):
                    z = (q[at:at + n, h].double() @ K.t() / math.sqrt(hd)).masked_fill(hide, float("-inf"))
                    l = torch.logsumexp(z, 1)
                    lse[at:at + n, h] = l
                    out[at:at + n, h] = torch.exp(z - l[:, None]) @ Vv
            at += n
        return out, lse
    probs = torch.zeros(case["rows"], dtype=torch.float64, device="cuda")
    V = case["vocab"]
    cols = torch.stack([s["temperature"].double(), s["top_k"].double(), s["top_p"].double(), s["min_p"].double(),
                        s["u"].double()], 1).tolist()
    for r in range(case["rows"]):
        T, k, p, lo, u = cols[r]
        x = s["logits"][r].double()
        if T == 0:
            probs[r] = 1.0
            continue
        w = torch.exp((x - x.max()) / T)
        w = w * (w >= 2.0 ** -40)
        big, who = torch.sort(w, descending=True, stable=True)
        n = int(k) if k > 0 else V
        mass = torch.cumsum(big[:n], 0)
        if p < 1:
            n = min(n, 1 + int((mass < p * mass[-1]).sum()))
        chosen = torch.zeros(V, dtype=torch.bool, device="cuda")
        chosen[who[:n]] = True
        w = w * (chosen & (w >= lo))
        c = torch.cumsum(w, 0)
        token = torch.searchsorted(c, u * c[-1], right=True).clamp(max=V - 1)
        probs[r] = w[token] / c[-1]
    return None, probs
