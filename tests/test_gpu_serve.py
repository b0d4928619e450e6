"""Serving operators against plain 64-bit forms (tests/serve_ref.py): page tables and row maps, the
K/V append, paged attention of chunks, sampling, and a run of them together."""
import math

import numpy as np
import pytest
import torch

import serve_ref as R

pytestmark = pytest.mark.gpu
PAGE = 16


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def status():
    from block_diffusion_drafter_forward_gb300 import serve_status
    return serve_status()


# ------------------------------------------------------------------------------ tables
TABLES = [
    # ctx, new, pages per sequence, free pages, begin, max_rows
    ([0], [1], 4, 4, 0, 1),
    ([15, 16, 17, 0], [1, 1, 0, 33], 4, 16, 3, 40),
    ([5], [0], 2, 2, 0, 7),
    ([0, 0, 0], [16, 15, 17], 2, 5, 1, 48),                      # exactly enough pages
    ([0, 0, 0], [16, 15, 17], 2, 4, 1, 48),                      # one page short: the last gets none
    ([3, 3, 3, 3], [4, 4, 4, 4], 1, 0, 0, 9),                    # rows for two only, no page needed
    ([0, 31, -1, 5, 2], [3, 2, 4, -2, 1], 2, 9, 0, 30),          # over capacity, negative lengths
    ([7, 0, 0], [0, 0, 0], 3, 3, 3, 0),
    ([0], [40000], 2500, 2500, 0, 40001),                        # one long prompt (several CTAs)
]


def tables_case(ctx, new, mpps, n_free, seed=0):
    g = torch.Generator().manual_seed(seed)
    nb = len(ctx)
    perm = torch.randperm(n_free + nb * mpps, generator=g).to(torch.int32)
    table = torch.full((nb, mpps), -7, dtype=torch.int32)
    at = n_free
    for s in range(nb):
        for i in range(min(mpps, max(0, -(-ctx[s] // PAGE)))):
            table[s, i] = perm[at]
            at += 1
    return table, perm[:n_free]


def check_tables(got, table, want):
    names = ("kv_lens", "row_starts", "row_seq", "row_index", "slots", "free_end")
    for name, g, w in zip(names, got, want[1:]):
        assert g.cpu().tolist() == list(w), name
    assert np.array_equal(table.cpu().numpy(), want[0]), "page_tables"


@pytest.mark.parametrize("ctx,new,mpps,n_free,begin,max_rows", TABLES)
def test_tables(ctx, new, mpps, n_free, begin, max_rows):
    from block_diffusion_drafter_forward_gb300 import _lib, extend_tables
    status()
    table, free = tables_case(ctx, new, mpps, n_free)
    want = R.tables(ctx, new, table, free.tolist(), begin, max_rows)
    t = table.cuda()
    got = extend_tables(i32(ctx), i32(new), t, free.cuda(), i32([begin]), max_rows)
    check_tables(got, t, want)
    cap = mpps * PAGE
    bad = any(c < 0 or n < 0 or c + n > cap for c, n in zip(ctx, new))
    asked = sum(n for c, n in zip(ctx, new) if c >= 0 and 0 <= n <= cap - c)
    short = asked > sum(np.diff(want[2]))
    assert status() == (_lib.DFLASH_DEV_BAD_CTX if bad else 0) | (_lib.DFLASH_DEV_NO_ROOM if short else 0)


@pytest.mark.parametrize("nb", [1, 31, 1024, 1025, 3000, 16384])
def test_tables_many_sequences_in_place(nb):
    """Lengths and the stack position written over the inputs, two steps in a row."""
    from block_diffusion_drafter_forward_gb300 import RowPlan, extend_tables
    r = np.random.RandomState(nb)
    ctx, mpps = r.randint(0, 60, nb).tolist(), 9
    total = [0, 0]
    news = [r.randint(0, 24, nb).tolist() for _ in range(2)]
    table, free = tables_case(ctx, news[0], mpps, 4 * nb, seed=nb)
    lens, pos, t, fr = i32(ctx), i32([0]), table.cuda(), free.cuda()
    rows = max(sum(n) for n in news) + 3
    e = lambda n: torch.empty(n, dtype=torch.int32, device="cuda")  # noqa: E731
    out = RowPlan(lens, e(nb + 1), e(rows), e(rows), e(rows), pos)
    begin = 0
    for new in news:
        want = R.tables(ctx, new, table, free.tolist(), begin, rows)
        got = extend_tables(lens, i32(new), t, fr, pos, rows, out=out)
        check_tables(got, t, want)
        table, ctx, begin = torch.tensor(want[0]), want[1], want[6][0]
    del total


# ------------------------------------------------------------------------------ append
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("nkv,hd,slots", [
    (1, 64, [0]), (3, 128, [5, 4, -1, 16, 47, 31]), (4, 128, list(range(3, 45))),
    (2, 64, list(range(8, 16)) + list(range(24, 32))), (2, 128, [40, 41, 42, 43, 44, 45, 46, 47, 0, 1, 2, 3, 4, 5, 6]),
    (1, 128, [8, 9, 10, 11, 12, 13, 14, 16]), (8, 64, list(range(47, -1, -1))), (5, 128, [-3] * 9),
])
def test_append(dtype, nkv, hd, slots):
    from block_diffusion_drafter_forward_gb300 import PagedKV
    status()
    g = torch.Generator().manual_seed(len(slots))
    n = len(slots)
    y = torch.randn(n, 3 * nkv * hd + 8, generator=g).to(dtype)     # rows of a wider tensor
    k, v = y[:, 8:8 + nkv * hd].view(n, nkv, hd), y[:, 8 + 2 * nkv * hd:].view(n, nkv, hd)
    pool = torch.randn(4, nkv, 2, 16 * hd, generator=g).to(dtype)   # a page whose stride is wider too
    wide = torch.zeros(4, nkv + 1, 2, 16 * hd, dtype=dtype, device="cuda")
    mine = wide[:, :nkv]
    mine.copy_(pool)
    yd = y.cuda()
    got = PagedKV(mine).append(yd[:, 8:8 + nkv * hd].view(n, nkv, hd), yd[:, 8 + 2 * nkv * hd:].view(n, nkv, hd), i32(slots))
    want = R.put(pool, k, v, slots)
    assert torch.equal(got.cpu(), want)
    assert bool((wide[:, nkv] == 0).all()) and status() == 0


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_pages_on_16_bytes_only(dtype):
    """A pool whose base and page stride are multiples of 16 bytes, not of 32: append, then attention."""
    from block_diffusion_drafter_forward_gb300 import PagedKV
    nkv, hd, P = 2, 128, 5
    off = 128 // torch.finfo(dtype).bits
    flat = torch.zeros(P * (32 * nkv * hd + off) + off, dtype=dtype, device="cuda")
    pool = flat[off:].as_strided((P, nkv, 2, 16 * hd), (32 * nkv * hd + off, 32 * hd, 16 * hd, 1), flat[off:].storage_offset())
    assert pool.data_ptr() % 32 == 16
    k, v = torch.randn(2, 70, nkv, hd, device="cuda").to(dtype)
    table = torch.tensor([[3, 1, 4, 0, 2]], dtype=torch.int32)
    slots = [int(table[0, i // 16]) * 16 + i % 16 for i in range(70)]
    kv = PagedKV(pool)
    kv.append(k, v, i32(slots))
    assert torch.equal(pool.cpu(), R.put(torch.zeros(P, nkv, 2, 16 * hd, dtype=dtype), k.cpu(), v.cpu(), slots))
    q = torch.randn(7, 8, hd, device="cuda").to(dtype)
    out, lse = kv.attend(q, table.cuda(), i32([70]), i32([0, 7]), 7, lse=torch.empty(7, 8, device="cuda"))
    check_attend(out, lse, R.attend(q, pool, table.cuda(), [70], [0, 7], True, 0, 1 / math.sqrt(hd)), slice(0, 7), hd)


def test_append_reports_slots_past_the_pages():
    from block_diffusion_drafter_forward_gb300 import PagedKV, _lib
    status()
    kv = PagedKV(torch.zeros(2, 1, 2, 16 * 64, device="cuda"))
    x = torch.ones(3, 1, 64, device="cuda")
    kv.append(x, x, i32([32, 2 ** 31 - 1, 7]))
    assert status() == _lib.DFLASH_DEV_BAD_PAGE and status() == 0
    assert int((kv.pool != 0).sum()) == 2 * 64


# ------------------------------------------------------------------------------ attend
def cache(ctx, new, nkv, hd, dtype, seed, gap=0):
    """Pages of sequences of ctx + new rows: rows past each end are NaN, as never-written rows may be."""
    g = torch.Generator().manual_seed(seed)
    lens = [c + n for c, n in zip(ctx, new)]
    pages = [-(-n // PAGE) for n in lens]
    total = sum(pages) + 2
    perm = torch.randperm(total, generator=g)
    mpps = max(pages) + 1
    table = torch.full((len(ctx), mpps), -5, dtype=torch.int32)
    pool = torch.full((total, nkv, 2, 16 * hd), float("nan"), dtype=dtype)
    d, at = torch.arange(hd), 0
    for s, n in enumerate(lens):
        table[s, :pages[s]] = perm[at:at + pages[s]].to(torch.int32)
        at += pages[s]
        for lp in range(pages[s]):
            r = min(PAGE, n - lp * PAGE)
            j = torch.arange(r)[:, None]
            pg = int(table[s, lp])
            pool[pg][:, 0, R.k_off(j, d, hd).reshape(-1)] = torch.randn(nkv, r * hd, generator=g).to(dtype)
            pool[pg][:, 1, R.v_off(j, d).reshape(-1)] = (torch.randn(nkv, r * hd, generator=g) + 0.3).to(dtype)
    starts = [gap]
    for n in new:
        starts.append(starts[-1] + n)
    return pool.cuda(), table.cuda(), lens, starts


def check_attend(got, lse, ref, rows, hd):
    """out: half a rounding step of the result, and of every probability where they go through the
    tensor cores as 16-bit operands; the sums in between are fp32."""
    o, l, spread, dots = (x[rows] for x in ref)
    half = torch.finfo(got.dtype).eps / 2
    # scores: a dot of hd products accumulated in fp32, then the exponent's rounding
    rel = 2.0 ** -24 * (hd + 8) * dots + 2.0 ** -20
    tol = half * o.abs() + (half + 2 * rel)[..., None] * spread + 1e-30 if got.dtype == torch.bfloat16 else \
        half * o.abs() + (2.0 ** -18 + 2 * rel)[..., None] * spread + 1e-30
    g = got[rows].double()
    assert torch.isfinite(g).all()
    worst = ((g - o).abs() / tol).max() if g.numel() else torch.tensor(0.0)
    assert worst <= 1, worst
    if lse is not None:
        seen = torch.isfinite(l)
        assert torch.equal(torch.isfinite(lse[rows]), seen)
        assert bool((lse[rows][~seen] == -math.inf).all())
        d = (lse[rows].double() - l).abs()[seen]
        assert bool((d <= (rel + 2.0 ** -22 * l.abs())[seen]).all()), d.max()


ATTEND = [
    # ctx, new, nh, nkv, hd, window, causal
    ([0], [1], 4, 1, 128, 0, True),
    ([4095], [1], 32, 4, 128, 0, True),
    ([0], [33], 8, 1, 128, 0, True),
    ([5, 0, 100, 31], [3, 0, 17, 1], 16, 2, 128, 0, True),          # a sequence without rows between others
    ([127, 128, 129, 255, 0], [1, 1, 1, 1, 1], 32, 4, 128, 0, True),
    ([300, 17], [16, 16], 32, 4, 128, 0, False),                      # the drafter's own mask
    ([700, 40, 2100], [20, 300, 5], 64, 8, 128, 48, True),          # window shorter than a chunk
    ([700, 40], [20, 129], 8, 1, 128, 1, True),                     # each row sees itself alone
    ([50, 60], [40, 30], 8, 8, 64, 0, True),                        # one query head per kv head
    ([0, 777], [250, 130], 8, 8, 128, 0, True),
    ([900, 3], [5, 70], 15, 3, 128, 0, True),                       # 5 query heads per kv head
    ([900, 3], [5, 70], 14, 2, 64, 100, True),
    ([33], [40], 128, 1, 64, 0, True),                              # 128 query heads on one kv head
    ([1000, 16], [2, 3], 48, 1, 128, 0, True),
    ([6000, 0, 2500, 90], [1, 600, 3, 64], 32, 4, 128, 0, True),    # single tokens, blocks and a prompt together
    ([5000, 4000], [1, 1], 8, 1, 64, 1000, True),
    ([0], [1500], 16, 2, 128, 0, True),
    ([0], [1500], 16, 2, 64, 333, False),
    # many chunks per CTA, so that both softmax streams go round the page rings many times
    ([30000, 28001, 31977, 25000, 29999, 27000], [1, 1, 2, 1, 1, 3], 32, 4, 128, 0, True),
    ([20000, 28001, 21977], [1, 30, 2], 32, 4, 64, 0, True),
    # single tokens among prompts: units whose second query tile is empty, long and short
    ([9000, 0, 7000, 20, 12000, 3, 8000], [1, 400, 1, 16, 1, 1, 90], 32, 4, 128, 0, True),
    ([3000] * 40, [1, 40, 2, 1, 1, 300, 1, 17] * 5, 32, 4, 128, 0, True),
]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("case", range(len(ATTEND)))
def test_attend(case, dtype):
    from block_diffusion_drafter_forward_gb300 import PagedKV
    status()
    ctx, new, nh, nkv, hd, window, causal = ATTEND[case]
    pool, table, lens, starts = cache(ctx, new, nkv, hd, dtype, case, gap=2)
    n = starts[-1] + 3                                              # rows before the first and behind the last sequence
    g = torch.Generator(device="cuda").manual_seed(case)
    wide = (torch.randn(n, nh + 2, hd, generator=g, device="cuda") * 1.5).to(dtype)
    q = wide[:, 1:1 + nh]                                           # rows of a wider tensor
    out = torch.full((n, nh + 1, hd), 7.0, dtype=dtype, device="cuda")
    lse = torch.full((n, nh), 7.0, device="cuda")
    scale = 0.5 if case % 5 == 4 else 1 / math.sqrt(hd)
    PagedKV(pool).attend(q, table, i32(lens), i32(starts), max(new), causal=causal, window=window,
                         scale=None if scale != 0.5 else 0.5, out=out[:, :nh], lse=lse)
    ref = R.attend(q, pool, table, lens, starts, causal, window, scale)
    rows = slice(2, starts[-1])
    check_attend(out[:, :nh], lse, ref, rows, hd)
    assert status() == 0
    untouched = torch.cat([out[:2], out[starts[-1]:]])
    assert bool((untouched == 7).all()) and bool((out[:, nh] == 7).all())
    assert bool((lse[:2] == 7).all()) and bool((lse[starts[-1]:] == 7).all())


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_attend_rows_without_keys(dtype):
    """kv_lens below the chunk (its first rows sit before key 0) and an empty cache: zeros, -inf."""
    from block_diffusion_drafter_forward_gb300 import PagedKV
    status()
    pool, table, _, _ = cache([0, 0], [20, 4], 2, 128, dtype, 3)
    lens, starts = [17, 0], [0, 20, 24]
    q = torch.randn(24, 16, 128, device="cuda").to(dtype)
    out, lse = PagedKV(pool).attend(q, table, i32(lens), i32(starts), 20, lse=torch.empty(24, 16, device="cuda"))
    check_attend(out, lse, R.attend(q, pool, table, lens, starts, True, 0, 1 / math.sqrt(128)), slice(0, 24), 128)
    assert bool((out[:3] == 0).all()) and bool((out[20:] == 0).all()) and bool((lse[20:] == -math.inf).all())
    assert status() == 0


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_attend_skips_sequences_out_of_range(dtype):
    from block_diffusion_drafter_forward_gb300 import PagedKV, _lib
    status()
    pool, table, lens, starts = cache([40, 50, 60], [2, 3, 4], 1, 128, dtype, 4)
    q = torch.randn(9, 8, 128, device="cuda").to(dtype)
    kv = PagedKV(pool)
    ref = R.attend(q, pool, table, lens, starts, True, 0, 1 / math.sqrt(128))
    for bad in (-1, table.shape[1] * PAGE + 1):
        out = torch.full((9, 8, 128), 7.0, dtype=dtype, device="cuda")
        kv.attend(q, table, i32([lens[0], bad, lens[2]]), i32(starts), 4, out=out)
        assert bool((out[2:5] == 7).all()) and status() == _lib.DFLASH_DEV_BAD_CTX
        check_attend(out, None, ref, slice(0, 2), 128)
        check_attend(out, None, ref, slice(5, 9), 128)
    kv.attend(q, table, i32(lens), i32([0, 2, 5, 10]), 4)           # past the rows of q
    assert status() == _lib.DFLASH_DEV_BAD_CTX
    broken = table.clone()
    broken[1, 1] = pool.shape[0]
    kv.attend(q, broken, i32(lens), i32(starts), 4)
    assert status() == _lib.DFLASH_DEV_BAD_PAGE


def test_attend_in_a_graph_and_on_a_stream():
    """Captured once, replayed with other lengths, tables and values; the same call on a side stream."""
    from block_diffusion_drafter_forward_gb300 import PagedKV
    sides = [([3000, 20, 0, 511], [1, 16, 30, 2]), ([10, 800, 2000, 37], [16, 3, 1, 29])]
    states = [cache(c, n, 4, 128, torch.bfloat16, 11 + i) for i, (c, n) in enumerate(sides)]
    P, mp = max(s[0].shape[0] for s in states), max(s[1].shape[1] for s in states)
    pool = torch.zeros(P, 4, 2, 16 * 128, dtype=torch.bfloat16, device="cuda")
    table = torch.zeros(4, mp, dtype=torch.int32, device="cuda")
    lens, starts = i32([0] * 4), i32([0] * 5)
    q = torch.randn(49, 32, 128, device="cuda").to(torch.bfloat16)
    out, lse = torch.zeros_like(q), torch.zeros(49, 32, device="cuda")
    kv = PagedKV(pool)

    def load(s):
        pool[:s[0].shape[0]].copy_(s[0])
        table[:, :s[1].shape[1]].copy_(s[1])
        lens.copy_(i32(s[2]))
        starts.copy_(i32(s[3]))

    load(states[0])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    kv.attend(q, table, lens, starts, 30, out=out, lse=lse, stream=side)
    side.synchronize()
    ref = [R.attend(q, s[0], s[1], s[2], s[3], True, 0, 1 / math.sqrt(128)) for s in states]
    check_attend(out, lse, ref[0], slice(0, 49), 128)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kv.attend(q, table, lens, starts, 30, out=out, lse=lse)
    for i in (1, 0, 1):
        load(states[i])
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        check_attend(out, lse, ref[i], slice(0, 49), 128)


def test_attend_whatever_the_hint_and_the_row_stride():
    """max_new picks the kernel and the way the work is found, not the result; a window past every
    length is none; rows of q any whole 16 bytes apart."""
    from block_diffusion_drafter_forward_gb300 import PagedKV
    ctx, new = [40, 0, 900, 7, 130] * 8, [1, 300, 17, 0, 64] * 8
    pool, table, lens, starts = cache(ctx, new, 2, 128, torch.bfloat16, 21)
    n = starts[-1]
    q = torch.randn(n, 16 * 128 + 8, device="cuda").to(torch.bfloat16).as_strided((n, 16, 128), (16 * 128 + 8, 128, 1))
    ref = R.attend(q, pool, table, lens, starts, True, 0, 1 / math.sqrt(128))
    kv = PagedKV(pool)
    for hint, window in ((0, 0), (1, 2 ** 31 - 1), (17, 0), (65, 2 ** 30), (300, 2 ** 32), (2 ** 33, 0)):
        out, lse = kv.attend(q, table, i32(lens), i32(starts), hint, window=window, lse=torch.empty(n, 16, device="cuda"))
        check_attend(out, lse, ref, slice(0, n), 128)


def test_attend_on_two_streams_at_once():
    """Calls that overlap have their own workspaces, eager and replayed, and give what they give alone."""
    from block_diffusion_drafter_forward_gb300 import PagedKV
    cases = [([9000] * 6, [1, 2, 16, 1, 1, 9], 0), ([0, 500, 3000], [900, 40, 200], 100)]
    calls, want = [], []
    for i, (ctx, new, window) in enumerate(cases):
        pool, table, lens, starts = cache(ctx, new, 4, 128, torch.bfloat16, 31 + i)
        q = torch.randn(starts[-1], 32, 128, device="cuda").to(torch.bfloat16)
        kv, args = PagedKV(pool), (q, table, i32(lens), i32(starts), max(new))
        calls.append(lambda out, st=None, kv=kv, a=args, w=window: kv.attend(*a, window=w, out=out, stream=st))
        want.append(calls[i](torch.zeros_like(q)).clone())
    graphs, outs = [], [torch.zeros_like(w) for w in want]
    for call, out in zip(calls, outs):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            call(out)
        graphs.append(g)
    streams = [torch.cuda.Stream() for _ in calls]
    for replay in (False, True):
        for o in outs:
            o.zero_()
        torch.cuda.synchronize()
        for _ in range(20):
            for call, g, out, st in zip(calls, graphs, outs, streams):
                if replay:
                    with torch.cuda.stream(st):
                        g.replay()
                else:
                    call(out, st)
        torch.cuda.synchronize()
        for o, w in zip(outs, want):
            assert torch.equal(o, w)


def test_pages_past_32_bits():
    """Page offsets of more than 2^31 elements: rows appended there come back through attend."""
    from block_diffusion_drafter_forward_gb300 import PagedKV
    nkv, hd, stride = 1, 64, 2 ** 30 + 8
    store = torch.empty(3 * stride, dtype=torch.bfloat16, device="cuda")
    far = PagedKV(store.as_strided((3, nkv, 2, 16 * hd), (stride, 2 * 16 * hd, 16 * hd, 1)))
    near = PagedKV.empty(3, nkv, hd)
    k, v = (torch.randn(40, nkv, hd, device="cuda").to(torch.bfloat16) for _ in range(2))
    slots = i32([(2 - i // 16) * 16 + i % 16 for i in range(40)])
    q = torch.randn(5, 4, hd, device="cuda").to(torch.bfloat16)
    got = []
    for kv in (far, near):
        kv.pool[0].zero_()
        kv.append(k, v, slots)
        got.append(kv.attend(q, i32([[2, 1, 0]]), i32([40]), i32([0, 5]), 5))
    assert torch.equal(far.pool, near.pool) and torch.equal(got[0], got[1])


def test_the_status_word_outlives_inference_mode():
    from block_diffusion_drafter_forward_gb300 import PagedKV, _lib, serve
    kept = dict(serve._status)
    serve._status.clear()
    try:
        with torch.inference_mode():
            kv = PagedKV(torch.zeros(2, 1, 2, 16 * 64, device="cuda"))
            kv.append(torch.ones(1, 1, 64, device="cuda"), torch.ones(1, 1, 64, device="cuda"), i32([32]))
        assert status() == _lib.DFLASH_DEV_BAD_PAGE and status() == 0
    finally:
        serve._status.clear()
        serve._status.update(kept)


# ------------------------------------------------------------------------------ sample
def check_sample(x, u, tokens, probs, T, k, p, lo, rows=None):
    xs, us = x.double().cpu().numpy(), u.double().cpu().numpy()
    col = lambda t, d: [d] * len(us) if t is None else t.cpu().double().tolist()  # noqa: E731
    Ts, ks, ps, los = col(T, 1.0), col(k, 0), col(p, 1.0), col(lo, 0.0)
    for r in range(len(us)):
        token, pr = R.sample(xs[r], us[r], Ts[r], int(ks[r]), ps[r], los[r])
        assert int(tokens[r]) == token, (r, int(tokens[r]), token, Ts[r], ks[r], ps[r], los[r], us[r])
        if probs is not None:  # rounded once from about 40 bits
            assert abs(float(probs[r]) - pr) <= 2.0 ** -23 * pr + 1e-12, (r, float(probs[r]), pr)


def logits(rows, V, dtype, seed, kind):
    g = torch.Generator(device="cuda").manual_seed(seed)
    if kind == "flat":
        return (torch.randn(rows, V, generator=g, device="cuda") * 0.3).to(dtype)
    if kind == "ties":
        return (torch.randint(-3, 4, (rows, V), generator=g, device="cuda") * 0.5).to(dtype)
    if kind == "equal":
        return torch.full((rows, V), -2.5, dtype=dtype, device="cuda")
    x = torch.randn(rows, V, generator=g, device="cuda") * 2
    x[:, :: max(1, V // 40)] += 8
    return x.to(dtype)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("kind", ["peaks", "flat", "ties", "equal"])
@pytest.mark.parametrize("V", [1, 2, 7, 63, 1000, 8191, 50257])
def test_sample(V, kind, dtype):
    """Every filter alone and together, per-row settings, over tiny, odd and large vocabularies."""
    from block_diffusion_drafter_forward_gb300 import sample
    sets = [(1.0, 0, 1.0, 0.0), (0.0, 5, 0.5, 0.1), (0.7, 1, 1.0, 0.0), (1.3, 5, 1.0, 0.0), (1.0, 40, 0.9, 0.0),
            (1.0, 0, 0.5, 0.0), (1.0, 0, 0.95, 0.0), (1.0, 0, 0.999, 0.05), (2.0, 0, 1.0, 0.2), (0.3, 1000, 0.8, 0.01),
            (1.0, 10 ** 9, 1.0, 0.0), (5.0, 300, 0.99, 0.0), (1.0, 0, 0.0, 0.0), (1.0, 0, 1e-6, 0.0), (1.0, 0, 1.0, 1.0),
            (1.0, 3, 0.7, 0.0)]
    rows = len(sets)
    g = torch.Generator(device="cuda").manual_seed(V)
    x = logits(rows, V, dtype, V, kind)
    u = torch.rand(rows, generator=g, device="cuda")
    T, p, lo = (torch.tensor([s[i] for s in sets], device="cuda") for i in (0, 2, 3))
    k = i32([s[1] for s in sets])
    probs = torch.empty(rows, device="cuda")
    tokens, _ = sample(x, u, T, k, p, lo, probs=probs)
    check_sample(x, u, tokens, probs, T, k, p, lo)
    check_sample(x, u, sample(x, u), None, None, None, None, None)                    # every option off
    check_sample(x, u, sample(x, u, top_p=p), None, None, None, p, None)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_sample_odd_rows_and_the_ends_of_u(dtype):
    """Rows of a wider tensor at odd addresses; u = 0, the largest below 1, 1 and NaN."""
    from block_diffusion_drafter_forward_gb300 import sample
    wide = logits(6, 1111, dtype, 5, "peaks")
    u = torch.tensor([0.0, 1 - 2.0 ** -24, 1.0, 0.5, float("nan"), -1.0], device="cuda")
    for at, V in ((0, 1111), (1, 1109), (3, 64), (7, 1)):
        x = wide[:, at:at + V]
        probs = torch.empty(6, device="cuda")
        tokens, _ = sample(x, u, probs=probs)
        check_sample(x, torch.nan_to_num(u), tokens, probs, None, None, None, None)
        p = torch.full((6,), 0.9, device="cuda")
        check_sample(x, torch.nan_to_num(u), sample(x, u, top_p=p), None, None, None, p, None)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_sample_rows_of_infinities_and_nan(dtype):
    from block_diffusion_drafter_forward_gb300 import sample
    inf, nan = math.inf, math.nan
    V = 300
    x = torch.randn(10, V, device="cuda").to(dtype)
    x[0] = -inf                                   # no candidate
    x[1] = nan
    x[2, 1:] = -inf                               # one candidate
    x[3, ::3] = inf                               # 100 equal largest
    x[4, ::2] = nan                               # half are not numbers
    x[5, 7] = inf
    x[6] = torch.finfo(dtype).min                 # the type's lowest value everywhere
    x[7, 5:] = torch.finfo(dtype).min
    x[8, 10:] = -inf                              # fewer candidates than k
    x[9, :150] = -0.0
    x[9, 150:] = 0.0
    u = torch.rand(10, device="cuda")
    for args in ((1.0, 0, 1.0, 0.0), (0.0, 0, 1.0, 0.0), (0.5, 20, 1.0, 0.0), (1.0, 0, 0.6, 0.0), (1.0, 150, 0.9, 0.1)):
        T, p, lo = (torch.full((10,), args[i], device="cuda") for i in (0, 2, 3))
        k = i32([args[1]] * 10)
        probs = torch.empty(10, device="cuda")
        tokens, _ = sample(x, u, T, k, p, lo, probs=probs)
        check_sample(x, u, tokens, probs, T, k, p, lo)
    y = torch.randn(5, V, device="cuda").to(dtype)
    T = torch.tensor([-1.0, inf, nan, 1e-38, 3e38], device="cuda")
    tokens, probs = sample(y, u[:5], T, probs=torch.empty(5, device="cuda"))
    assert tokens[:3].tolist() == [-1] * 3 and probs[:3].tolist() == [0.0] * 3
    check_sample(y[3:], u[3:5], tokens[3:], probs[3:], T[3:], None, None, None)
    lo = torch.full((5,), 1.5, device="cuda")     # above the largest weight
    assert sample(y, u[:5], min_p=lo).tolist() == [-1] * 5


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_sample_top_p_at_its_borders(dtype):
    """p a rounding of fp32 away from the mass of a prefix, a tenth of the mass past it: whether the
    next logit stays is decided by the 8th digit of the row's total."""
    from block_diffusion_drafter_forward_gb300 import sample
    rows, V = 256, 20000
    g = torch.Generator(device="cuda").manual_seed(12)
    x = (torch.randn(rows, V, generator=g, device="cuda") * 3).to(dtype)
    p = []
    for row in x.double().cpu().numpy():
        w = np.exp(np.sort(row)[::-1] - row.max())
        c = np.cumsum(np.where(w >= 2.0 ** -40, w, 0.0))
        p.append(c[np.searchsorted(c, (0.85 + 0.1 * len(p) / rows) * c[-1])] / c[-1])
    p = torch.tensor(p, device="cuda").float()
    u, probs = torch.rand(rows, generator=g, device="cuda"), torch.empty(rows, device="cuda")
    tokens, _ = sample(x, u, top_p=p, probs=probs)
    check_sample(x, u, tokens, probs, None, None, p, None)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_sample_u_at_its_borders(dtype):
    """u a rounding of fp32 away from the mass ahead of a token, most of it small weights."""
    from block_diffusion_drafter_forward_gb300 import sample
    rows, V = 256, 20000
    g = torch.Generator(device="cuda").manual_seed(13)
    x = (torch.randn(rows, V, generator=g, device="cuda") * 2).to(dtype)
    x[:, 777] = 9.0
    u, rng = [], np.random.default_rng(5)
    for row in x.double().cpu().numpy():
        w = np.exp(row - row.max())
        c = np.cumsum(np.where(w >= 2.0 ** -40, w, 0.0))
        while True:  # (further than 1e-11 from the border, which the definition leaves open)
            i = int(rng.integers(V))
            v = float(np.float32(c[i] / c[-1]))
            if abs(v * c[-1] - c[i]) > 1e-11 * c[-1] and 0 < v < 1:
                break
        u.append(v)
    u, probs = torch.tensor(u, device="cuda"), torch.empty(rows, device="cuda")
    tokens, _ = sample(x, u, probs=probs)
    check_sample(x, u, tokens, probs, None, None, None, None)


def test_sample_rows_past_32_bits():
    from block_diffusion_drafter_forward_gb300 import sample
    x = logits(3, 1000, torch.bfloat16, 7, "peaks")
    far = torch.empty(2 * (2 ** 30 + 24) + 1000, dtype=torch.bfloat16, device="cuda").as_strided((3, 1000), (2 ** 30 + 24, 1))
    far.copy_(x)
    u = torch.rand(3, device="cuda")
    a, b = (sample(t, u, probs=torch.empty(3, device="cuda")) for t in (x, far))
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_sample_large_vocabulary_and_a_graph():
    from block_diffusion_drafter_forward_gb300 import sample
    for dtype, V in ((torch.float32, 376000), (torch.bfloat16, 752000), (torch.bfloat16, 262144)):
        x = logits(4, V, dtype, 9, "peaks")
        u = torch.rand(4, device="cuda")
        p, k = torch.tensor([1.0, 0.9, 0.3, 0.99], device="cuda"), i32([0, 0, 500, 30])
        tokens = torch.empty(4, dtype=torch.int32, device="cuda")
        probs = torch.empty(4, device="cuda")
        sample(x, u, top_k=k, top_p=p, tokens=tokens, probs=probs)
        check_sample(x, u, tokens, probs, None, k, p, None)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        sample(x, u, top_k=k, top_p=p, tokens=tokens, probs=probs)
    x.copy_(logits(4, V, dtype, 10, "flat"))
    u.uniform_()
    graph.replay()
    torch.cuda.synchronize()
    check_sample(x, u, tokens, probs, None, k, p, None)


# ------------------------------------------------------------------------------ together
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_steps_of_a_batch(dtype):
    """Prompts, then two steps of new tokens: tables, append, attention and a draw per sequence, all on
    the device, against the dense computation over every row so far."""
    from block_diffusion_drafter_forward_gb300 import PagedKV, extend_tables, sample
    status()
    nb, nkv, nh, hd, mpps, V = 5, 2, 16, 128, 12, 997
    g = torch.Generator(device="cuda").manual_seed(1)
    kv = PagedKV.empty(64, nkv, hd, dtype)
    kv.pool.fill_(float("nan"))
    table = torch.full((nb, mpps), -1, dtype=torch.int32, device="cuda")
    free, at, lens = torch.randperm(64, device="cuda").to(torch.int32), i32([0]), i32([0] * nb)
    head = torch.randn(nh * hd, V, generator=g, device="cuda").to(dtype)
    past = [(torch.zeros(0, nkv, hd, dtype=dtype, device="cuda"),) * 2 for _ in range(nb)]
    for new in ([1, 100, 0, 37, 16], [1, 1, 50, 1, 16], [3, 1, 1, 1, 1]):
        T = sum(new)
        plan = extend_tables(lens, i32(new), table, free, at, T + 4)
        qkv = torch.randn(T + 4, nh + 2 * nkv, hd, generator=g, device="cuda").to(dtype)
        kv.append(qkv[:, nh:nh + nkv], qkv[:, nh + nkv:], plan.slots)
        out = kv.attend(qkv[:, :nh], table, plan.kv_lens, plan.row_starts, max(new))
        assert bool((out[T:] == 0).all())
        i = 0
        for s, n in enumerate(new):
            K, Vv = (torch.cat([a, b[i:i + n]]) for a, b in zip(past[s], (qkv[:, nh:nh + nkv], qkv[:, nh + nkv:])))
            past[s] = (K, Vv)
            kk, vv = (x.double().repeat_interleave(nh // nkv, 1) for x in (K, Vv))
            sc = torch.einsum("ihd,jhd->hij", qkv[i:i + n, :nh].double(), kk) / math.sqrt(hd)
            far = torch.arange(len(K) - n, len(K), device="cuda")[:, None] < torch.arange(len(K), device="cuda")
            p = torch.softmax(sc.masked_fill(far, -math.inf), 2)
            want, spread = torch.einsum("hij,jhd->ihd", p, vv), torch.einsum("hij,jhd->ihd", p, vv.abs())
            half = torch.finfo(dtype).eps / 2
            tol = half * want.abs() + (half + 2.0 ** -14) * spread
            assert bool(((out[i:i + n].double() - want).abs() <= tol).all())
            i += n
        z = out[:T].reshape(T, nh * hd) @ head
        u = torch.rand(T, generator=g, device="cuda")
        k = torch.full((T,), 50, dtype=torch.int32, device="cuda")
        check_sample(z, u, sample(z, u, top_k=k), None, None, k, None, None)
        lens, at = plan.kv_lens, plan.free_end
    assert status() == 0


def test_plan_feeds_the_drafter_writer_and_attend_reads_its_pool():
    """extend_tables' rows into Drafter.write_ctx_kv_batch, and attention over the drafter's own pages
    (Drafter.kv_pages) against its rows read back."""
    from block_diffusion_drafter_forward_gb300 import Drafter, extend_tables
    from synth import CONFIGS, make_weights
    from synth.torch_io import upload_weights
    status()
    cfg = CONFIGS["small_gqa4_bf16"]
    d = Drafter(cfg, upload_weights(make_weights(cfg, 3)), num_pages=40, max_batch=3, max_pages_per_seq=10)
    ctx, new = [0, 0, 0], [40, 1, 77]
    table = torch.full((3, 10), -1, dtype=torch.int32, device="cuda")
    plan = extend_tables(i32(ctx), i32(new), table, torch.randperm(40, device="cuda").to(torch.int32), i32([0]), sum(new))
    g = torch.Generator(device="cuda").manual_seed(2)
    taps = torch.randn(sum(new), cfg.n_taps * cfg.target_hidden, generator=g, device="cuda").to(torch.bfloat16)
    d.write_ctx_kv_batch(taps, plan.row_index, plan.row_seq, plan.row_index, table)
    assert d.device_status() == 0
    q = torch.randn(sum(new), cfg.n_q_heads, cfg.head_dim, generator=g, device="cuda").to(torch.bfloat16)
    for layer in range(cfg.n_layers):
        kv = d.kv_pages(layer)
        out, lse = kv.attend(q, table, plan.kv_lens, plan.row_starts, max(new), lse=torch.empty(sum(new), cfg.n_q_heads, device="cuda"))
        ref = R.attend(q, kv.pool, table, new, plan.row_starts.tolist(), True, 0, 1 / math.sqrt(cfg.head_dim))
        check_attend(out, lse, ref, slice(0, sum(new)), cfg.head_dim)
    assert status() == 0
