"""Calls of the tree, rotary and 8-bit operators that their documentation allows and single-call tests do not
make: hints that are wrong, very many sequences, units of a chunk or two, calls at once, captured steps."""
import math
import random

import pytest
import torch

import verify_ref as V
from test_gpu_serve import cache, check_attend
from test_gpu_verify import BF, F32, cache8, i32, plan_of, some_tree, status

pytestmark = pytest.mark.gpu
PAGE = 16


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


def plain8(q, kv, table, lens, starts, scale=None, **kw):
    return V.attend(q, lambda s, m: V.rows8(kv.pool, table[s], m), lens, starts, scale or 1 / math.sqrt(q.shape[2]), **kw)


@pytest.mark.parametrize("nh,nkv,hd", [(8, 1, 128), (64, 1, 64), (128, 1, 128), (3, 3, 64), (17, 1, 128), (10, 2, 128)])
def test_attend_in_8_bits_whatever_the_hint(nh, nkv, hd):
    """The hint picks the form only: none, less or more than the chunks, and more heads than a unit of 16 rows holds."""
    status()
    ctx, new = [700, 0, 33, 2000], [1, 40, 16, 3]
    kv, table, lens, starts = cache8(ctx, new, nkv, hd, nh)
    parents, plan = plan_of(new, lens, starts, nh, 64)
    q = torch.randn(sum(new), nh, hd, device="cuda").to(BF)
    refs = plain8(q, kv, table, lens, starts), plain8(q, kv, table, lens, starts, parents=parents)
    for hint in (0, 1, 2, 40, 100000):
        for tree, ref in zip((None, plan), refs):
            out, lse = kv.attend(q, table, i32(lens), i32(starts), hint, tree=tree, lse=torch.empty(sum(new), nh, device="cuda"))
            check_attend(out, lse, ref, slice(0, sum(new)), hd)
    assert status() == 0


@pytest.mark.parametrize("hd", [64, 128])
@pytest.mark.parametrize("form", ["blocks", "ragged", "trees", "tokens"])
def test_attend_in_8_bits_many_short_sequences(form, hd):
    """Units of one, two or a few chunks, several to a CTA, so that streams have segments without work between others."""
    status()
    r = random.Random(hd + len(form))
    nb = 700 if form == "tokens" else 300
    if form == "blocks":
        ctx, new = [60] * nb, [16] * nb
    elif form == "tokens":
        ctx, new = [r.choice((0, 1, 15, 16, 175, 176, 177, 400)) for _ in range(nb)], [1] * nb
    else:
        ctx, new = [r.choice((0, 1, 100, 111, 112, 113, 250, 600)) for _ in range(nb)], [r.choice((0, 1, 2, 16, 17, 40)) for _ in range(nb)]
    kv, table, lens, starts = cache8(ctx, new, 2, hd, nb + hd)
    parents, plan = plan_of(new, lens, starts, 1, 64) if form == "trees" else (None, None)
    q = torch.randn(starts[-1], 16, hd, device="cuda").to(BF)
    ref = plain8(q, kv, table, lens, starts, parents=parents)
    for _ in range(3):
        out, lse = kv.attend(q, table, i32(lens), i32(starts), max(new), tree=plan, lse=torch.empty(starts[-1], 16, device="cuda"))
        check_attend(out, lse, ref, slice(0, starts[-1]), hd)
    assert status() == 0


@pytest.mark.parametrize("new", [1, 5])
def test_attend_in_8_bits_the_most_sequences(new):
    """16384 sequences share two pages' rows: the plan at its limit; one more is refused."""
    from block_diffusion_drafter_forward_gb300 import DflashError
    status()
    nb, nh = 16384, 8
    kv, table, lens, _ = cache8([20], [new], 1, 64, new)
    q = torch.randn(nb * new, nh, 64, device="cuda").to(BF)
    tables, starts = table.expand(nb, -1).contiguous(), i32(list(range(0, nb * new + 1, new)))
    out = kv.attend(q, tables, i32(lens * nb), starts, new)
    for s in (0, 1, 7777, nb - 1):
        part = q[s * new:(s + 1) * new]
        check_attend(out[s * new:(s + 1) * new], None, plain8(part, kv, table, lens, [0, new]), slice(0, new), 64)
    with pytest.raises(DflashError, match="16384"):
        kv.attend(q, torch.cat([tables, table]), i32(lens * (nb + 1)), i32([0] * (nb + 2)), new)
    assert status() == 0


def test_attend_peaked_rows_in_8_bits():
    """Rows whose weights lie on a few keys, over many chunks and segments, again and again: a page's values in the
    wrong place or at the wrong time would show in them, where an even row would hide them."""
    nkv, hd, L = 2, 128, 3000
    for new in (1, 16, 100):
        nb = 24
        kv, table, lens, starts = cache8([L - new] * nb, [new] * nb, nkv, hd, new)
        rows = [V.rows8(kv.pool, table[s], L) for s in range(nb)]
        g = torch.Generator().manual_seed(new)
        q = torch.empty(nb * new, 8, hd)
        for s in range(nb):
            for i in range(new):
                j = int(torch.randint(0, L - new, (1,), generator=g))
                for h in range(8):
                    k = rows[s][0][j, h // 4]
                    q[s * new + i, h] = (k / k.norm() * 40).float()
        q = q.to(BF).cuda()
        ref = plain8(q, kv, table, lens, starts, scale=1.0)
        for _ in range(8):
            check_attend(kv.attend(q, table, i32(lens), i32(starts), new, scale=1.0), None, ref, slice(0, nb * new), hd)


def test_trees_on_two_streams_at_once():
    from block_diffusion_drafter_forward_gb300 import PagedKV, draft_tree
    sides = [([3000, 20, 0, 511], [20, 64, 30, 2]), ([10, 800, 2000, 37], [64, 3, 1, 29])]
    streams = [torch.cuda.Stream() for _ in sides]
    calls = []
    for i, (ctx, new) in enumerate(sides):
        pool, table, lens, starts = cache(ctx, new, 4, 128, BF, 21 + i)
        parents = [p for s, n in enumerate(new) for p in some_tree(n, s)]
        q = torch.randn(sum(new), 32, 128, device="cuda").to(BF)
        ref = V.attend(q, V.rows16(pool, table), lens, starts, 1 / math.sqrt(128), parents=parents)
        calls.append((PagedKV(pool), q, table, i32(lens), i32(starts), i32(parents), ref, torch.zeros_like(q)))
    torch.cuda.synchronize()
    for _ in range(6):
        for st, (kv, q, table, lens, starts, parents, _, out) in zip(streams, calls):
            plan = draft_tree(parents, lens, starts, 64, stream=st)
            kv.attend(q, table, lens, starts, 64, tree=plan, out=out, stream=st)
    torch.cuda.synchronize()
    for kv, q, _, _, _, _, ref, out in calls:
        check_attend(out, None, ref, slice(0, q.shape[0]), 128)


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
def test_a_tree_verified_and_kept_in_a_graph(kind):
    """Tables, tree, rotary positions, append, attention and the move of the branch, captured once and replayed
    with other trees, lengths and branches."""
    from block_diffusion_drafter_forward_gb300 import PagedKV, QuantKV, Rope, RowPlan, TreePlan, draft_tree, extend_tables
    nkv, nh, hd, nb, nodes, cap = 2, 8, 64, 3, 20, 8
    g = torch.Generator(device="cuda").manual_seed(3)
    kv = QuantKV.empty(nb * cap, nkv, hd) if kind == "e4m3" else PagedKV.empty(nb * cap, nkv, hd)
    kv.pool.fill_(255) if kind == "e4m3" else kv.pool.fill_(float("nan"))
    rope = Rope(hd, 1e4, interleaved=True)
    ctx, new, table, pos, held = i32([0] * nb), i32([0] * nb), i32([[-1] * cap] * nb), i32([0]), i32([0] * nb)
    free, rows = i32(torch.randperm(nb * cap).tolist()), nb * nodes
    e = lambda *n: torch.empty(n, dtype=torch.int32, device="cuda")  # noqa: E731
    plan = RowPlan(e(nb), e(nb + 1), e(rows), e(rows), e(rows), pos)
    tree = TreePlan(e(rows), torch.empty(rows, 1, dtype=torch.int64, device="cuda"))
    parents, path, path_lens = i32([-1] * rows), i32([[0] * nodes] * nb), i32([0] * nb)
    q, k, v = (torch.zeros(rows, h, hd, dtype=BF, device="cuda") for h in (nh, nkv, nkv))
    qr, kr, out = torch.empty_like(q), torch.empty_like(k), torch.zeros_like(q)

    def step():
        extend_tables(ctx, new, table, free, pos, rows, out=plan, held_pages=held)
        draft_tree(parents, plan.kv_lens, plan.row_starts, nodes, out=tree)
        rope.rotate(q, tree.positions, k=k, out=qr, k_out=kr)
        kv.append(kr, v, plan.slots)
        kv.attend(qr, table, plan.kv_lens, plan.row_starts, nodes, tree=tree, out=out)
        kv.keep(table, ctx, path, path_lens)
    status()
    step()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    r = random.Random(5)
    past, lens = [(torch.zeros(0, nkv, hd, dtype=torch.float64, device="cuda"),) * 2 for _ in range(nb)], [0] * nb
    for _ in range(5):
        sizes = [r.randint(0, nodes) for _ in range(nb)]
        trees = [some_tree(n, r.random()) for n in sizes]
        paths = []
        for t in trees:
            at, branch = r.randrange(len(t)) if t else -1, []
            while at >= 0:
                branch.append(at)
                at = t[at]
            paths.append(branch[::-1])
        flat = [p for t in trees for p in t]
        for t, x in ((ctx, lens), (new, sizes), (path_lens, [len(p) for p in paths]), (parents, flat + [-1] * (rows - len(flat))),
                     (path, [p + [0] * (nodes - len(p)) for p in paths])):
            t.copy_(i32(x))
        for t in (q, k, v):
            t.copy_(torch.randn(t.shape, generator=g, device="cuda").to(BF))
        graph.replay()
        i = 0
        for s, n in enumerate(sizes):
            depth, see = V.tree(trees[s])
            assert tree.positions[i:i + n].tolist() == [lens[s] + d for d in depth]
            fresh = [V.quantise(x[i:i + n].cpu())[0].cuda() if kind == "e4m3" else x[i:i + n].double() for x in (kr, v)]
            if n:
                K, Vv = (torch.cat([a, b]).repeat_interleave(nh // nkv, 1) for a, b in zip(past[s], fresh))
                hide = torch.cat([torch.zeros(n, lens[s], dtype=torch.bool), ~torch.tensor(see)], 1).cuda()
                p = (torch.einsum("ihd,jhd->hij", qr[i:i + n].double(), K) / math.sqrt(hd)).masked_fill(hide, -math.inf).softmax(2)
                want, spread = torch.einsum("hij,jhd->ihd", p, Vv), torch.einsum("hij,jhd->ihd", p, Vv.abs())
                # P and the output rounded to bf16, half a step each; fp32 sums and exponentials of scores of a few units
                assert bool(((out[i:i + n].double() - want).abs() <= 2.0 ** -8 * (spread + want.abs()) + 1e-4 * spread + 1e-6).all())
            past[s] = tuple(torch.cat([a, b[paths[s]]]) for a, b in zip(past[s], fresh))
            lens[s] += len(paths[s])
            i += n
    assert status() == 0


@pytest.mark.parametrize("dtype", [BF, F32])
def test_two_sequences_on_one_page_and_rows_twice(dtype):
    """Reads may share pages: two sequences over the same prefix, and a slot read twice."""
    kv, table, lens, starts = cache8([100], [3], 1, 64, 9)
    q = torch.randn(6, 4, 64, device="cuda").to(dtype)
    both = kv.attend(q, torch.cat([table, table]), i32(lens * 2), i32([0, 3, 6]), 3)
    check_attend(both, None, plain8(q, kv, torch.cat([table, table]), lens * 2, [0, 3, 6]), slice(0, 6), 64)
    slot = int(table[0, 0]) * PAGE
    k, v = kv.read(i32([slot, slot, slot + 1, slot]), dtype=dtype)
    assert torch.equal(k[0], k[1]) and torch.equal(k[0], k[3]) and torch.equal(v[0], v[3])


def test_rotate_a_padded_step():
    """extend_tables' row_index holds -1 behind the step's rows: those rows are rotated by -1 like any position, the
    others as without them; positions at both ends of int32."""
    from block_diffusion_drafter_forward_gb300 import Rope
    rope = Rope(64, 1e4)
    q = torch.randn(5, 2, 64, device="cuda")
    pos = i32([7, 2 ** 31 - 1, -2 ** 31, -1, -1])
    got = rope.rotate(q, pos)
    ref, size = V.rotate(q.double(), pos.cpu(), rope.turns.tolist(), 1.0, False)
    assert bool(((got.double() - ref).abs() <= 10 * 2.0 ** -24 * size + 2.0 ** -24 * ref.abs()).all())
    assert torch.equal(got[:1], rope.rotate(q[:1], pos[:1]))
