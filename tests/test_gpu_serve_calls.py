"""Calls of the serving operators that their documentation allows and single-call tests do not make:
streams that share the status word, steps that go back, lengths and hints at the ends of their range."""
import math

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


def test_the_status_word_is_read_and_cleared_at_once():
    """While one stream sets a bit all along and reads, another's bit arrives whenever it was set.  (A torch
    operation on the word would be a load and a store: bits set between them were lost.)"""
    from block_diffusion_drafter_forward_gb300 import PagedKV, _lib, extend_tables, serve
    status()
    word = serve._status[torch.cuda.current_device()]
    kv = PagedKV(torch.zeros(2, 1, 2, PAGE * 64, device="cuda"))
    one = torch.ones(1, 1, 64, device="cuda")
    bad = i32([2 * PAGE])
    version = word._version
    kv.append(one, one, bad)
    assert status() == _lib.DFLASH_DEV_BAD_PAGE and status() == 0
    assert word._version == version
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    full = (i32([0]), i32([1]), i32([[0]]), i32([0]), i32([1]), 1)
    for _ in range(100):
        kv.append(one, one, bad, stream=side)
        seen = 0
        for _ in range(3):
            extend_tables(*full)
            seen |= status()
        side.synchronize()
        assert seen | status() == _lib.DFLASH_DEV_BAD_PAGE | _lib.DFLASH_DEV_NO_ROOM


def tables_held(ctx, new, table, free, begin, max_rows, held):
    """extend_tables with the pages held, row by row: (table, held, kv_lens, slots, free_end), all lists."""
    table, held = [list(t) for t in table], list(held)
    cap = len(table[0])
    at, rows, room, kv, slots = begin, 0, True, [], []
    for s, (c, n) in enumerate(zip(ctx, new)):
        if c < 0 or n < 0 or c + n > cap * PAGE or not -(-c // PAGE) <= held[s] <= cap:
            kv.append(c)
            continue
        need = max(0, -(-(c + n) // PAGE) - held[s])
        room = room and at + need <= len(free) and rows + n <= max_rows
        if not room:
            kv.append(c)
            continue
        for _ in range(need):
            table[s][held[s]] = free[at]
            held[s] += 1
            at += 1
        slots += [table[s][i // PAGE] * PAGE + i % PAGE for i in range(c, c + n)]
        rows += n
        kv.append(c + n)
    return table, held, kv, slots + [-1] * (max_rows - rows), at


@pytest.mark.parametrize("nb,block", [(1, 16), (7, 16), (33, 16), (200, 5), (300, 40)])
def test_tables_of_sequences_that_go_back(nb, block):
    """Steps of verification, of which a random part of each block stays: no page is given twice, a sequence
    never takes one while it has one, the stack holds out, and rows that stay keep their place."""
    from block_diffusion_drafter_forward_gb300 import extend_tables
    status()
    g = torch.Generator().manual_seed(nb)
    r = lambda lo, hi, n=nb: torch.randint(lo, hi + 1, (n,), generator=g).tolist()  # noqa: E731
    steps, cap = 12, -(-12 * (block + 1) // PAGE) + 1
    ctx, table, held = [0] * nb, [[-1] * cap for _ in range(nb)], [0] * nb
    free = torch.randperm(nb * cap, generator=g).tolist()
    begin, most, max_rows = 0, [0] * nb, nb * block + 3
    t_table, t_free, t_begin, t_held = i32(table), i32(free), i32([0]), i32(held)
    places = [[] for _ in range(nb)]
    for step in range(steps):
        new = r(0, block) if step % 3 == 2 else [block] * nb
        want = tables_held(ctx, new, table, free, begin, max_rows, held)
        plan = extend_tables(i32(ctx), i32(new), t_table, t_free, t_begin, max_rows, held_pages=t_held)
        table, held, kv, slots, begin = want
        assert t_table.tolist() == table and t_held.tolist() == held and plan.kv_lens.tolist() == kv
        assert plan.slots.tolist() == slots and plan.free_end.tolist() == [begin]
        t_begin = plan.free_end
        most = [max(a, -(-b // PAGE)) for a, b in zip(most, kv)]
        assert held == most                                  # no more than the sequence ever needed at once
        owned = [p for row, h in zip(table, held) for p in row[:h]]
        assert len(set(owned)) == len(owned) == begin
        for s in range(nb):
            places[s] = places[s][:ctx[s]] + slots[sum(new[:s]):sum(new[:s + 1])]
            assert places[s] == [table[s][i // PAGE] * PAGE + i % PAGE for i in range(kv[s])]
        stay = r(0, block)
        ctx = [c + min(a, n) for c, a, n in zip(ctx, stay, new)]
    assert status() == 0


@pytest.mark.parametrize("nb", [5, 2000])
def test_pages_held_out_of_range_and_short_stacks(nb):
    """Held pages below what the rows fill or past the table: no rows, a status bit, the others served; the
    stack or the rows run out in the middle; lengths and the stack's position written in place."""
    from block_diffusion_drafter_forward_gb300 import RowPlan, _lib, extend_tables
    status()
    g = torch.Generator().manual_seed(nb)
    cap = 6
    for n_free, max_rows in ((4 * nb, 40 * nb), (nb, 40 * nb), (4 * nb, 9 * nb), (0, 5000)):
        ctx = torch.randint(0, 60, (nb,), generator=g).tolist()
        new = torch.randint(0, 37, (nb,), generator=g).tolist()
        held = [-(-c // PAGE) + x for c, x in zip(ctx, torch.randint(0, 3, (nb,), generator=g).tolist())]
        held = [min(h, cap) for h in held]
        held[1], held[3] = cap + 1, -1
        ctx[4], held[4] = 17, 1
        perm = torch.randperm(nb * cap + n_free, generator=g).tolist()
        table = [[perm[s * cap + i] if i < held[s] else -1 for i in range(cap)] for s in range(nb)]
        free = perm[nb * cap:]
        want = tables_held(ctx, new, table, free, 0, max_rows, held)
        t_ctx, t_table, t_held, t_pos = i32(ctx), i32(table), i32(held), i32([0])
        e = lambda n: torch.empty(n, dtype=torch.int32, device="cuda")  # noqa: E731
        out = RowPlan(t_ctx, e(nb + 1), e(max_rows), e(max_rows), e(max_rows), t_pos)
        extend_tables(t_ctx, i32(new), t_table, i32(free), t_pos, max_rows, out=out, held_pages=t_held)
        assert (t_table.tolist(), t_held.tolist(), t_ctx.tolist(), out.slots.tolist(), t_pos.item()) == want
        short = sum(n for n in want[2]) - sum(ctx) < sum(n for s, n in enumerate(new) if s not in (1, 3, 4))
        assert status() == _lib.DFLASH_DEV_BAD_CTX | (_lib.DFLASH_DEV_NO_ROOM if short else 0)


def test_a_block_verified_twice_in_a_graph():
    """Tables with pages held, append and attention captured together and replayed as a sequence goes on,
    back and on: the rows that stay are attended to as if the rejected ones had never been."""
    from block_diffusion_drafter_forward_gb300 import PagedKV, RowPlan, extend_tables
    nkv, hd, nb, block, cap = 2, 128, 3, 16, 8
    g = torch.Generator(device="cuda").manual_seed(3)
    bf = torch.bfloat16
    kv = PagedKV.empty(nb * cap, nkv, hd)
    kv.pool.fill_(float("nan"))
    ctx, new, table, pos, held = i32([0] * nb), i32([block] * nb), i32([[-1] * cap] * nb), i32([0]), i32([0] * nb)
    free = i32(torch.randperm(nb * cap).tolist())
    rows = nb * block
    e = lambda n: torch.empty(n, dtype=torch.int32, device="cuda")  # noqa: E731
    plan = RowPlan(e(nb), e(nb + 1), e(rows), e(rows), e(rows), pos)
    q, k, v = (torch.empty(rows, h, hd, dtype=bf, device="cuda") for h in (8, nkv, nkv))
    out = torch.zeros_like(q)

    def step():
        extend_tables(ctx, new, table, free, pos, rows, out=plan, held_pages=held)
        kv.append(k, v, plan.slots)
        kv.attend(q, table, plan.kv_lens, plan.row_starts, block, out=out)
    status()
    for t in (q, k, v):
        t.zero_()
    new.zero_()
    step()  # (no rows: nothing is taken)
    new.fill_(block)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    keys, vals, lens = [torch.zeros(0, nkv, hd, dtype=bf, device="cuda") for _ in range(nb)], None, [0] * nb
    vals = [x.clone() for x in keys]
    for stay in ([16, 3, 0], [1, 15, 7], [16, 16, 16], [0, 2, 5], [9, 9, 9]):
        for t in (q, k, v):
            t.copy_(torch.randn(t.shape, generator=g, device="cuda").to(bf))
        ctx.copy_(i32(lens))
        graph.replay()
        for s in range(nb):
            at = slice(s * block, (s + 1) * block)
            K, V = (torch.cat([old[s], fresh[at]]).double().repeat_interleave(4, 1) for old, fresh in ((keys, k), (vals, v)))
            sc = torch.einsum("ihd,jhd->hij", q[at].double(), K) / math.sqrt(hd)
            i, j = torch.arange(block, device="cuda")[:, None], torch.arange(K.shape[0], device="cuda")[None]
            p = sc.masked_fill(j > lens[s] + i, -math.inf).softmax(2)
            ref = torch.einsum("hij,jhd->ihd", p, V)
            spread = torch.einsum("hij,jhd->ihd", p, V.abs())
            # P and the output rounded to bf16, half a step each; fp32 sums and exponentials of scores of a few tens
            assert bool(((out[at].double() - ref).abs() <= 2.0 ** -8 * (spread + ref.abs()) + 1e-4 * spread + 1e-6).all())
            keys[s], vals[s] = (torch.cat([old[s], fresh[at][:stay[s]]]) for old, fresh in ((keys, k), (vals, v)))
            lens[s] += stay[s]
    assert status() == 0 and int(pos) == int(held.sum()) <= nb * cap


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("kv_lens,starts", [
    ([20, -1, 30], [0, 2, 2, 5]),          # a negative length, of a sequence without rows
    ([20, 1000, 30], [0, 2, 2, 5]),        # and one past its table
    ([20, 16, 30], [0, 2, 9, 9]),          # rows past q, of which the first five have a sequence of their own
    ([20, 16, 30], [3, 5, 1, 3]),          # starts that fall: the second has none, the third has rows 1 and 2
])
def test_every_sequence_out_of_range_is_reported(kv_lens, starts, dtype):
    from block_diffusion_drafter_forward_gb300 import PagedKV, _lib
    status()
    g = torch.Generator(device="cuda").manual_seed(1)
    kv = PagedKV(torch.randn(9, 1, 2, PAGE * 64, generator=g, device="cuda").to(dtype))
    q = torch.randn(5, 2, 64, generator=g, device="cuda").to(dtype)
    table = torch.arange(9, dtype=torch.int32, device="cuda").view(3, 3)
    kv.attend(q, table, i32(kv_lens), i32(starts), 3)
    assert status() == _lib.DFLASH_DEV_BAD_CTX


def test_rows_on_pages_that_are_none_are_reported():
    """A table entry, or an id on the stack, that is no page: its rows have no slot, and a status bit says so."""
    from block_diffusion_drafter_forward_gb300 import _lib, extend_tables
    status()
    for table, free, slots in (([[-7, -1], [3, -1]], [4, 5], [-1, -1, 3 * PAGE + 5, 3 * PAGE + 6]), ([[2 ** 27, 0], [3, 0]], [4, 5], [-1, -1, 53, 54]),
                               ([[1, -1], [3, -1]], [-2, 5], [21, 22, 53, 54])):
        t = i32(table)
        plan = extend_tables(i32([5, 5]), i32([2, 2]), t, i32(free), i32([0]), 4)
        assert plan.slots.tolist() == slots and plan.row_index.tolist() == [5, 6, 5, 6] and t.tolist() == table
        assert status() == (_lib.DFLASH_DEV_BAD_PAGE if -1 in slots else 0)
    plan = extend_tables(i32([15]), i32([2]), i32([[1, -1]]), i32([-2]), i32([0]), 2)
    assert plan.slots.tolist() == [31, -1] and status() == _lib.DFLASH_DEV_BAD_PAGE


def test_sizes_and_hints_that_32_bits_would_cut_are_refused():
    from block_diffusion_drafter_forward_gb300 import DflashError, PagedKV, sample
    kv = PagedKV(torch.zeros(2, 1, 2, PAGE * 64, device="cuda"))
    q, table = torch.zeros(1, 1, 64, device="cuda"), i32([[0, 1]])
    for kw in (dict(window=-2 ** 32), dict(window=-2 ** 32 + 7), dict(max_new=-2 ** 32), dict(max_new=-1)):
        with pytest.raises(DflashError, match="attend"):
            kv.attend(q, table, i32([1]), i32([0, 1]), **{"max_new": 1, **kw})
    long = torch.empty(1, 2 ** 32 + 5, dtype=torch.bfloat16, device="cuda")  # never read
    with pytest.raises(ValueError, match="logits of a row: 4294967301 are too many"):
        sample(long, torch.zeros(1, device="cuda"))
