"""Drafted trees (masks, attention, kept rows), rotary positions and pages in 8 bits against plain 64-bit
forms (tests/verify_ref.py), and a run of them together."""
import math
import random

import pytest
import torch

import serve_ref as R
import verify_ref as V
from test_gpu_serve import cache, check_attend

pytestmark = pytest.mark.gpu
PAGE = 16
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def status():
    from block_diffusion_drafter_forward_gb300 import serve_status
    return serve_status()


def some_tree(n, seed, chain=False):
    r = random.Random(seed)
    return [-1 if i == 0 else i - 1 if chain else r.choice((-1, i - 1, r.randint(0, i - 1), max(0, i - 3))) for i in range(n)]


# ------------------------------------------------------------------------------ rotary positions
ROTATE = [
    # rows, q heads, k heads, head dim, rotary dim, interleaved
    (1, 1, 0, 16, 16, False), (1, 32, 4, 128, 128, False), (3, 8, 1, 64, 32, True), (17, 5, 5, 96, 48, False),
    (64, 64, 8, 128, 128, True), (700, 15, 3, 128, 64, False), (5, 2, 1, 512, 512, True), (2, 3, 2, 512, 16, False),
    (1500, 1, 1, 64, 64, False), (9, 300, 100, 32, 32, True), (4097, 2, 1, 80, 80, False),
]


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("case", range(len(ROTATE)))
def test_rotate(case, dtype):
    from block_diffusion_drafter_forward_gb300 import Rope
    rows, nh, nk, hd, rd, inter = ROTATE[case]
    g = torch.Generator(device="cuda").manual_seed(case)
    yarn = (32.0, 8192.0, 32.0, 1.0) if case % 3 == 1 else None
    rope = Rope(rd, theta=1e4 if case % 2 else 1e6, linear=4.0 if case % 3 == 2 else 1.0, yarn=yarn, interleaved=inter)
    wide = torch.randn(rows, (nh + nk) * hd + 16, generator=g, device="cuda").to(dtype)
    q, k = wide[:, 8:8 + nh * hd].view(rows, nh, hd), wide[:, 8 + nh * hd:8 + (nh + nk) * hd].view(rows, nk, hd)
    far = (100, 10 ** 6, 2 ** 31 - 1)[case % 3]
    pos = torch.randint(-far - 1 if case % 4 == 3 else 0, far, (rows,), generator=g, device="cuda").to(torch.int32)
    before = wide.clone()
    for inverse in (False, True):
        got = rope.rotate(q, pos, k=k if nk else None, inverse=inverse)
        for y, x in zip(got if nk else (got,), (q, k)):
            ref, size = V.rotate(x.double(), pos.cpu(), rope.turns.tolist(), rope.mscale, inter, inverse)
            # the angle to 2^-24 half turns, sine and cosine to 2^-23 of 1, the scale and two products and their sum to
            # 2^-24 each: 10 times 2^-24 of the two magnitudes, and the result's own rounding
            tol = 10 * 2.0 ** -24 * size + torch.finfo(dtype).eps / 2 * ref.abs()
            assert bool(((y.double() - ref).abs() <= tol).all())
    assert torch.equal(wide, before)
    # in place: the same bits, and nothing beside the heads
    want = rope.rotate(q, pos, k=k if nk else None)
    want = want if nk else (want,)
    got = rope.rotate(q, pos, k=k if nk else None, out=q, k_out=k if nk else None)
    assert torch.equal(q, want[0]) and (not nk or torch.equal(k, want[1]))
    assert torch.equal(wide[:, :8], before[:, :8]) and torch.equal(wide[:, 8 + (nh + nk) * hd:], before[:, 8 + (nh + nk) * hd:])


def test_rotate_takes_gradients_back():
    """The inverse is the transpose: <y', R x> = <R^T y', x>, and R^T y' agrees with differences of <y', R x>."""
    from block_diffusion_drafter_forward_gb300 import Rope
    for inter in (False, True):
        rope = Rope(48, 1e4, yarn=(4.0, 64.0, 32.0, 1.0), interleaved=inter)
        x, w = torch.randn(2, 33, 3, 64, device="cuda")
        pos = torch.randint(0, 5000, (33,), device="cuda").to(torch.int32)
        back = rope.rotate(w, pos, inverse=True)
        a, b = (w.double() * rope.rotate(x, pos).double()).sum(), (back.double() * x.double()).sum()
        # 6336 products of terms to 10 2^-24 of two magnitudes of a few units each
        assert abs(float(a - b)) <= 6336 * 10 * 2.0 ** -24 * 4
        for _ in range(20):
            at = tuple(random.randrange(s) for s in x.shape)
            step = torch.zeros_like(x)
            step[at] = 1.0
            d = (w.double() * (rope.rotate(x + step, pos).double() - rope.rotate(x - step, pos).double())).sum() / 2
            # (the map is linear: a step of 1 has no error of its own; 64 outputs of its head to 10 2^-24 of some 12)
            assert abs(float(d) - float(back[at])) <= 64 * 10 * 2.0 ** -24 * 12


def test_rotate_one_row_like_many_and_in_a_graph():
    """A row's result does not depend on the rows beside it (the split of heads does); a captured call takes new values."""
    from block_diffusion_drafter_forward_gb300 import Rope
    rope = Rope(128, 1e6)
    q, pos = torch.randn(9000, 8, 128, device="cuda").to(BF), torch.arange(9000, device="cuda").to(torch.int32)
    many = rope.rotate(q, pos)
    for r in (0, 1, 4567, 8999):
        assert torch.equal(rope.rotate(q[r:r + 1], pos[r:r + 1]), many[r:r + 1])
    assert torch.equal(rope.rotate(q[:0], pos[:0]), q[:0])
    out = torch.empty_like(q)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    rope.rotate(q, pos, out=out, stream=side)
    side.synchronize()
    assert torch.equal(out, many)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        rope.rotate(q, pos, out=out)
    pos.copy_(torch.flip(pos, (0,)))
    graph.replay()
    assert torch.equal(out, rope.rotate(q, pos))


def test_rotate_refuses():
    from block_diffusion_drafter_forward_gb300 import DflashError, Rope
    rope = Rope(64)
    q, pos = torch.zeros(2, 3, 64, device="cuda"), i32([0, 1])
    with pytest.raises(DflashError):
        rope.rotate(torch.zeros(2, 3, 48, device="cuda"), pos)          # a head below the rotated dims
    for bad in (dict(k=q.to(BF)), dict(k=q[:1]), dict(k_out=q), dict(out=q[:, :2]), dict(k=q, k_out=q[:1]), dict(out=q.to(BF))):
        with pytest.raises(ValueError):
            rope.rotate(q, pos, **bad)
    with pytest.raises(ValueError):
        rope.rotate(q, pos[:1])
    with pytest.raises(ValueError):
        rope.rotate(q, pos.long())
    with pytest.raises(ValueError):
        rope.rotate(q.transpose(1, 2), pos)
    with pytest.raises(ValueError, match="the table is on cpu"):
        Rope(64, device="cpu").rotate(q, pos)


# ------------------------------------------------------------------------------ trees
@pytest.mark.parametrize("sizes,most", [([1], 1), ([16], 16), ([64, 0, 65, 1, 512], 512), ([3] * 300, 3), ([31, 64], 64), ([128, 127], 200), ([0, 0], 4)])
def test_draft_tree(sizes, most):
    from block_diffusion_drafter_forward_gb300 import draft_tree
    status()
    parents = [[7, 8]] + [some_tree(n, i, chain=i % 3 == 2) for i, n in enumerate(sizes)] + [[5, -9, 3]]
    starts = [2]
    for n in sizes:
        starts.append(starts[-1] + n)
    kv = [n + (i * 37) % 5000 for i, n in enumerate(sizes)]
    flat = [p for t in parents for p in t]
    plan = draft_tree(i32(flat), i32(kv), i32(starts), most)
    n_words = -(-most // 64)
    pos, masks = [-1, -1], [[0] * n_words] * 2
    for t, c, n in zip(parents[1:-1], kv, sizes):
        depth, see = V.tree(t)
        pos += [c - n + d for d in depth]
        masks += V.words(see, n_words)
    assert plan.positions.tolist() == pos + [-1] * 3 and plan.masks.tolist() == masks + [[0] * n_words] * 3
    assert status() == 0


def test_draft_tree_reports_what_is_none():
    from block_diffusion_drafter_forward_gb300 import _lib, draft_tree
    status()
    plan = draft_tree(i32([-1, 1, 0, 5, -2]), i32([15]), i32([0, 5]), 64)     # a node its own parent, one behind it, below -1
    assert plan.positions.tolist() == [10, 10, 11, 10, 10] and plan.masks[:, 0].tolist() == [1, 2, 5, 8, 16]
    assert status() == _lib.DFLASH_DEV_BAD_TREE
    plan = draft_tree(i32([-1] * 70), i32([100, 100]), i32([0, 65, 70]), 64)  # more nodes than the masks hold
    assert plan.positions.tolist() == [-1] * 65 + [95] * 5 and not plan.masks[:65].any()
    assert status() == _lib.DFLASH_DEV_BAD_TREE
    plan = draft_tree(i32([-1] * 5), i32([2, 9]), i32([0, 3, 5]), 64)         # fewer rows in the cache than nodes
    assert plan.positions.tolist() == [-1] * 3 + [7] * 2 and status() == _lib.DFLASH_DEV_BAD_CTX
    for starts in ([0, 4, 2], [0, 2, 6], [-1, 2, 5]):
        draft_tree(i32([-1] * 5), i32([9, 9]), i32(starts), 64)
        assert status() == _lib.DFLASH_DEV_BAD_CTX


TREES = [
    # ctx, nodes, nh, nkv, hd, window
    ([0], [1], 4, 1, 128, 0), ([4096], [32], 32, 4, 128, 0), ([0], [64], 8, 1, 64, 0), ([5, 0, 100, 31], [3, 0, 17, 1], 16, 2, 128, 0),
    ([127, 128, 129, 250, 16], [1, 16, 40, 63, 64], 32, 4, 128, 0),         # trees across chunk and page edges
    ([700, 40, 2100], [20, 200, 65], 64, 8, 128, 256), ([1000, 0], [512, 300], 8, 8, 128, 0), ([900, 3], [5, 70], 15, 3, 64, 128),
    ([6000, 0, 2500, 90], [33, 64, 1, 47], 32, 4, 128, 0), ([30000, 28001, 31977, 25000], [16, 2, 31, 64], 32, 4, 128, 0),
    ([60, 61, 62, 63, 64, 65] * 6, [3, 9, 30, 2, 1, 64] * 6, 8, 1, 128, 64), ([5000, 4000], [1, 2], 8, 1, 64, 1000),
    ([100, 3000], [130, 200], 16, 16, 128, 0), ([20], [40], 128, 1, 64, 0),
]


def plan_of(new, lens, starts, seed, most=None):
    from block_diffusion_drafter_forward_gb300 import draft_tree
    parents = [0] * starts[0] + [p for i, n in enumerate(new) for p in some_tree(n, 100 * seed + i, chain=(seed + i) % 5 == 4)]
    return parents, draft_tree(i32(parents), i32(lens), i32(starts), most or max(new))


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("case", range(len(TREES)))
def test_attend_trees(case, dtype):
    from block_diffusion_drafter_forward_gb300 import PagedKV
    status()
    ctx, new, nh, nkv, hd, window = TREES[case]
    pool, table, lens, starts = cache(ctx, new, nkv, hd, dtype, case, gap=2)
    parents, plan = plan_of(new, lens, starts, case)
    n = starts[-1]
    q = (torch.randn(n, nh, hd, generator=torch.Generator(device="cuda").manual_seed(case), device="cuda") * 1.5).to(dtype)
    out, lse = torch.full((n, nh, hd), 7.0, dtype=dtype, device="cuda"), torch.full((n, nh), 7.0, device="cuda")
    scale = 0.5 if case % 5 == 4 else 1 / math.sqrt(hd)
    PagedKV(pool).attend(q, table, i32(lens), i32(starts), max(new), window=window, scale=scale, out=out, lse=lse, tree=plan)
    ref = V.attend(q, V.rows16(pool, table), lens, starts, scale, window=window, parents=parents)
    check_attend(out, lse, ref, slice(2, n), hd)
    assert status() == 0 and bool((out[:2] == 7).all()) and bool((lse[:2] == 7).all())


@pytest.mark.parametrize("dtype", [BF, F32])
def test_attend_a_chain_is_causal_attention(dtype):
    """A tree that is one chain sees what a causal chunk sees: the same to its roundings, whatever the hint."""
    from block_diffusion_drafter_forward_gb300 import PagedKV, draft_tree
    new = [16, 1, 64]
    pool, table, lens, starts = cache([333, 20, 1000], new, 2, 128, dtype, 5)
    plan = draft_tree(i32([p for n in new for p in [-1] + list(range(n - 1))]), i32(lens), i32(starts), 300)
    q = torch.randn(81, 16, 128, device="cuda").to(dtype)
    kv = PagedKV(pool)
    want = kv.attend(q, table, i32(lens), i32(starts), 64)
    for hint in (0, 64, 500):
        got = kv.attend(q, table, i32(lens), i32(starts), hint, tree=plan)
        assert float((got.double() - want.double()).abs().max()) <= 2.0 ** -7 * 8


@pytest.mark.parametrize("dtype", [BF, F32])
def test_attend_masks_of_the_callers_own(dtype):
    """Masks that hide everything (no context: zeros and -inf), that see later rows, and bits past the tree."""
    from block_diffusion_drafter_forward_gb300 import PagedKV, TreePlan, _lib
    status()
    for c in (0, 200):
        pool, table, lens, starts = cache([c], [70], 1, 128, dtype, 6)
        g = torch.Generator().manual_seed(c)
        see = torch.rand(70, 70, generator=g) < 0.3
        see[3] = see[69] = False
        bits = V.words([r.tolist() + [True] * 58 for r in see], 2)
        plan = TreePlan(i32([c] * 70), torch.tensor(bits, dtype=torch.int64, device="cuda"))
        q = torch.randn(70, 8, 128, device="cuda").to(dtype)
        out, lse = PagedKV(pool).attend(q, table, i32(lens), i32(starts), 70, tree=plan, lse=torch.empty(70, 8, device="cuda"))
        K, Vv = (x.repeat_interleave(8, 1) for x in R.rows_of(pool, table[0], c + 70))
        hide = torch.zeros(70, c + 70, dtype=torch.bool, device="cuda")
        hide[:, c:] = ~see.cuda()
        sc = torch.einsum("ihd,jhd->hij", q.double(), K) / math.sqrt(128)
        dots = torch.einsum("ihd,jhd->hij", q.double().abs(), K.abs()).amax(2).t() / math.sqrt(128)
        sc = sc.masked_fill(hide, -math.inf)
        l = torch.logsumexp(sc, 2)
        p = torch.exp(sc - torch.where(l > -math.inf, l, 0.0)[..., None])
        check_attend(out, lse, (torch.einsum("hij,jhd->ihd", p, Vv), l.t(), torch.einsum("hij,jhd->ihd", p, Vv.abs()), dots), slice(0, 70), 128)
        if c == 0:
            assert bool((out[[3, 69]] == 0).all()) and bool((lse[[3, 69]] == -math.inf).all())
    assert status() == 0
    # more rows than the masks have bits: the sequence is skipped
    pool, table, lens, starts = cache([40, 8], [65, 3], 1, 128, dtype, 7)
    plan = TreePlan(i32([0] * 68), torch.full((68, 1), -1, dtype=torch.int64, device="cuda"))
    out = torch.full((68, 8, 128), 7.0, dtype=dtype, device="cuda")
    PagedKV(pool).attend(torch.randn(68, 8, 128, device="cuda").to(dtype), table, i32(lens), i32(starts), 65, tree=plan, out=out)
    assert status() == _lib.DFLASH_DEV_BAD_CTX and bool((out[:65] == 7).all()) and not bool((out[65:] == 7).any())


@pytest.mark.parametrize("kind", ["bf16", "f32", "e4m3"])
def test_attend_trees_with_positions_of_the_callers_own(kind):
    """Positions far behind and far before the sequence: the window hides context by them, own rows go by the mask."""
    from block_diffusion_drafter_forward_gb300 import PagedKV, TreePlan
    status()
    for n, ctx in ((2, 200), (40, 200)):
        if kind == "e4m3":
            kv, table, lens, starts = cache8([ctx], [n], 1, 128, n)
            rows = V.rows8(kv.pool, table[0], ctx + n)
        else:
            pool, table, lens, starts = cache([ctx], [n], 1, 128, BF if kind == "bf16" else F32, n)
            kv, rows = PagedKV(pool), R.rows_of(pool, table[0], ctx + n)
        pos = [(5, ctx + 3, ctx + 70, ctx + 100000, 2 ** 31 - 1, -7)[i % 6] for i in range(n)]
        see = [[(i * 7 + j) % 3 > 0 for j in range(n)] for i in range(n)]
        plan = TreePlan(i32(pos), torch.tensor(V.words(see, 1), dtype=torch.int64, device="cuda"))
        q = torch.randn(n, 8, 128, device="cuda").to(F32 if kind == "f32" else BF)
        out, lse = kv.attend(q, table, i32(lens), i32(starts), n, window=64, tree=plan, lse=torch.empty(n, 8, device="cuda"))
        K, Vv = (x.cuda().repeat_interleave(8, 1) for x in rows)
        hide = torch.tensor([[max(ctx, p) - j >= 64 for j in range(ctx)] + [not x for x in see[i]] for i, p in enumerate(pos)], device="cuda")
        sc = torch.einsum("ihd,jhd->hij", q.double(), K) / math.sqrt(128)
        dots = torch.einsum("ihd,jhd->hij", q.double().abs(), K.abs()).amax(2).t() / math.sqrt(128)
        sc = sc.masked_fill(hide, -math.inf)
        l = torch.logsumexp(sc, 2)
        p = torch.exp(sc - torch.where(l > -math.inf, l, 0.0)[..., None])
        check_attend(out, lse, (torch.einsum("hij,jhd->ihd", p, Vv), l.t(), torch.einsum("hij,jhd->ihd", p, Vv.abs()), dots), slice(0, n), 128)
    assert status() == 0


def test_attend_trees_refuses():
    from block_diffusion_drafter_forward_gb300 import DflashError, PagedKV, QuantKV, TreePlan
    kv = PagedKV(torch.zeros(2, 1, 2, PAGE * 64, device="cuda"))
    q, table, plan = torch.zeros(2, 1, 64, device="cuda"), i32([[0, 1]]), TreePlan(i32([0, 0]), torch.ones(2, 1, dtype=torch.int64, device="cuda"))
    args = (q, table, i32([2]), i32([0, 2]), 2)
    with pytest.raises(DflashError, match="hide ancestors"):
        kv.attend(*args, window=63, tree=plan)
    kv.attend(*args, window=64, tree=plan)
    for bad in (plan._replace(positions=i32([0])), plan._replace(masks=plan.masks.int()), plan._replace(masks=plan.masks[:1]),
                plan._replace(masks=plan.masks[:, 0]), plan._replace(positions=plan.positions.cpu())):
        with pytest.raises(ValueError):
            kv.attend(*args, tree=bad)
    with pytest.raises(DflashError, match="mask_words"):
        kv.attend(*args, tree=plan._replace(masks=torch.ones(2, 9, dtype=torch.int64, device="cuda")))
    with pytest.raises(ValueError, match="float32"):
        kv.attend(q.to(BF), *args[1:])
    quant = QuantKV(torch.zeros(2, 1, 32 * 64 + 32, dtype=torch.uint8, device="cuda"))
    with pytest.raises(ValueError, match="bfloat16"):
        quant.attend(q.half(), *args[1:])
    with pytest.raises(ValueError):
        QuantKV(torch.zeros(2, 1, 32 * 96 + 32, dtype=torch.uint8, device="cuda"))
    with pytest.raises(ValueError):
        QuantKV(torch.zeros(2, 1, 32 * 64 + 32, device="cuda"))


# ------------------------------------------------------------------------------ kept rows
@pytest.mark.parametrize("kind", ["bf16", "f32", "e4m3"])
@pytest.mark.parametrize("nkv,hd", [(1, 64), (3, 128), (8, 128)])
def test_keep(kind, nkv, hd):
    """Branches of every length, among them none, whole chunks, and rows that move over a page's edge."""
    from block_diffusion_drafter_forward_gb300 import PagedKV, QuantKV
    status()
    r = random.Random(nkv)
    ctx = [0, 5, 16, 31, 100, 47, 0, 3]
    new = [1, 30, 64, 17, 512, 40, 9, 20]
    paths = [[0], [0, 3, 4, 29], [], list(range(17)), sorted(r.sample(range(512), 300)), [39], list(range(9)), [1, 2, 15, 16, 17, 18, 19]]
    paths[2] = sorted(r.sample(range(64), 20))
    paths[5] = []
    pages = [-(-(c + n) // PAGE) for c, n in zip(ctx, new)]
    perm = torch.randperm(sum(pages) + 2, generator=torch.Generator().manual_seed(1)).to(torch.int32)
    table, at = torch.full((8, max(pages)), -1, dtype=torch.int32), 0
    for s, n in enumerate(pages):
        table[s, :n] = perm[at:at + n]
        at += n
    g = torch.Generator().manual_seed(2)
    if kind == "e4m3":
        pool = torch.randint(0, 256, (len(perm), nkv, 32 * hd + 32), generator=g).to(torch.uint8)
        es, tile = 1, 32 * hd + 32
    else:
        pool = torch.randn(len(perm), nkv, 2, 16 * hd, generator=g).to(BF if kind == "bf16" else F32)
    d = torch.arange(hd)
    want = pool.clone()
    for s, path in enumerate(paths):
        for i, x in enumerate(path):
            (a, ja), (b, jb) = ((int(table[s, (ctx[s] + y) // PAGE]), (ctx[s] + y) % PAGE) for y in (x, i))
            if kind == "e4m3":
                want[b, :, V.k8(jb, d)] = pool[a, :, V.k8(ja, d)]
                want[b, :, 16 * hd + V.v8(jb, d)] = pool[a, :, 16 * hd + V.v8(ja, d)]
                for side in (0, 16):
                    want[b, :, 32 * hd + side + jb] = pool[a, :, 32 * hd + side + ja]
            else:
                want[b, :, 0, R.k_off(jb, d, hd)] = pool[a, :, 0, R.k_off(ja, d, hd)]
                want[b, :, 1, R.v_off(jb, d)] = pool[a, :, 1, R.v_off(ja, d)]
    longest = max(map(len, paths)) + 1
    padded = [p + [-77] * (longest - len(p)) for p in paths]
    # pages in a tensor of more heads, so that their stride is wider
    wide = torch.zeros(len(perm), nkv + 1, *pool.shape[2:], dtype=pool.dtype, device="cuda")
    mine = wide[:, :nkv]
    mine.copy_(pool)
    kv = QuantKV(mine) if kind == "e4m3" else PagedKV(mine)
    got = kv.keep(table.cuda(), i32(ctx), i32(padded), i32([len(p) for p in paths]))
    assert got.data_ptr() == mine.data_ptr()
    assert torch.equal(mine.cpu().view(torch.uint8), want.view(torch.uint8)) and bool((wide[:, nkv] == 0).all())
    assert status() == 0


def test_keep_leaves_what_it_refuses():
    from block_diffusion_drafter_forward_gb300 import PagedKV, _lib
    status()
    pool = torch.randn(6, 2, 2, PAGE * 64, device="cuda")
    table = i32([[0, 1, 2], [3, 4, 5]])
    for ctx, path, lens, flag in (([0, 0], [[1, 1], [0, 0]], [2, 0], "BAD_TREE"), ([0, 0], [[-1, 1], [0, 0]], [2, 0], "BAD_TREE"),
                                  ([0, 0], [[5, 4], [0, 0]], [2, 0], "BAD_TREE"), ([0, 0], [[1, 3], [0, 0]], [3, 0], "BAD_TREE"),
                                  ([0, 0], [[1, 3], [0, 0]], [-1, 0], "BAD_TREE"), ([-1, 0], [[1, 3], [0, 0]], [2, 0], "BAD_CTX"),
                                  ([46, 0], [[1, 2], [0, 0]], [2, 0], "BAD_CTX"), ([0, 0], [[1, 2 ** 31 - 1], [0, 0]], [2, 0], "BAD_CTX")):
        kv = PagedKV(pool.clone())
        kv.keep(table, i32(ctx), i32(path), i32(lens))
        assert torch.equal(kv.pool, pool) and status() == getattr(_lib, "DFLASH_DEV_" + flag), (ctx, path, lens)
    kv = PagedKV(pool.clone())
    kv.keep(i32([[0, 6, 2], [3, -1, 5]]), i32([10, 0]), i32([[2, 10, 25], [1, 2, 33]]), i32([3, 3]))
    want = pool.clone()
    d = torch.arange(64)
    for p, a, q, b in ((0, 12, 0, 10), (2, 3, 0, 12), (3, 1, 3, 0), (3, 2, 3, 1), (5, 1, 3, 2)):  # (row 20 lies on no page)
        want[q, :, 0, R.k_off(b, d, 64)] = pool[p, :, 0, R.k_off(a, d, 64)]
        want[q, :, 1, R.v_off(b, d)] = pool[p, :, 1, R.v_off(a, d)]
    assert torch.equal(kv.pool, want) and status() == _lib.DFLASH_DEV_BAD_PAGE
    assert torch.equal(kv.keep(table, i32([0, 0]), i32([[], []]).view(2, 0), i32([0, 0])), want) and status() == 0


# ------------------------------------------------------------------------------ pages in 8 bits
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("nkv,hd,slots", [
    (1, 64, [0]), (3, 128, [5, 4, -1, 16, 47, 31]), (4, 128, list(range(3, 45))), (3, 64, list(range(8, 16)) + list(range(24, 32))),
    (2, 128, [40, 41, 42, 43, 44, 45, 46, 47, 0, 1, 2, 3, 4, 5, 6]), (1, 128, [8, 9, 10, 11, 12, 13, 14, 16]), (8, 64, list(range(47, -1, -1))),
    (5, 128, [-3] * 9), (5, 64, [-1] + list(range(16, 32)) + [-1, 2]),
])
def test_append_and_read_in_8_bits(dtype, nkv, hd, slots):
    from block_diffusion_drafter_forward_gb300 import QuantKV
    status()
    g = torch.Generator().manual_seed(len(slots))
    n = len(slots)
    y = torch.randn(n, 3 * nkv * hd + 8, generator=g) * torch.exp2(torch.randint(-20, 20, (n, 1), generator=g).float())
    y[:, ::37] *= 300
    y = y.to(dtype)                                                   # rows of a wider tensor
    k, v = y[:, 8:8 + nkv * hd].view(n, nkv, hd), y[:, 8 + 2 * nkv * hd:].view(n, nkv, hd)
    pool = torch.randint(0, 256, (4, nkv, 32 * hd + 32), generator=g).to(torch.uint8)
    wide = torch.zeros(4, nkv + 1, 32 * hd + 32, dtype=torch.uint8, device="cuda")
    mine = wide[:, :nkv]
    mine.copy_(pool)
    yd = y.cuda()
    kv = QuantKV(mine)
    kv.append(yd[:, 8:8 + nkv * hd].view(n, nkv, hd), yd[:, 8 + 2 * nkv * hd:].view(n, nkv, hd), i32(slots))
    assert torch.equal(mine.cpu(), V.put8(pool, k, v, slots))
    assert bool((wide[:, nkv] == 0).all()) and status() == 0
    for out in (BF, F32):
        into = torch.full((2, n, nkv + 1, hd), 7.0, dtype=out, device="cuda")
        got = kv.read(i32(slots), dtype=out, k=into[0, :, :nkv], v=into[1, :, :nkv])
        for x, want in zip(got, (k, v)):
            want = V.quantise(want)[0]
            want[torch.tensor(slots) < 0] = 0
            assert torch.equal(x.cpu().double(), want)
        assert bool((into[:, :, nkv] == 7).all())
    assert status() == 0


@pytest.mark.parametrize("dtype", [BF, F32])
def test_rows_at_the_ends_of_8_bits(dtype):
    """Zeros, the largest and smallest numbers, ties, infinities and NaN, -0, and every power between."""
    from block_diffusion_drafter_forward_gb300 import QuantKV
    big = float(torch.finfo(dtype).max)
    rows = [torch.zeros(64), torch.full((64,), big), torch.full((64,), 2.0 ** -133), torch.full((64,), -0.0),
            torch.tensor([math.inf, -math.inf, math.nan, 1.0] * 16), torch.tensor([math.nan] * 64), torch.tensor([big, 1e30, -1e36, 0.5] * 16),
            torch.tensor([V.code_value(c) for c in range(64)]), torch.tensor([V.code_value(c) for c in range(64, 127)] + [448.0]),
            torch.tensor([(V.code_value(c) + V.code_value(c + 1)) / 2 for c in range(62)] + [448.0, -448.0]),
            torch.tensor([(V.code_value(c) + V.code_value(c + 1)) / 2 for c in range(62, 124)] + [448.0, -0.0])]
    rows += [torch.linspace(-1, 1, 64) * 2.0 ** k * m for k in range(-130, 126, 3) for m in (1.75, 1.7578125)]
    n = len(rows) // 2 * 2
    x = torch.stack(rows[:n]).to(dtype).view(n // 2, 2, 64)
    kv = QuantKV.empty(-(-n // PAGE), 2, 64)
    slots = list(range(n // 2))
    kv.append(x.cuda(), x.flip(0).cuda(), i32(slots))
    for out in (BF, F32):
        for got, want in zip(kv.read(i32(slots), dtype=out), (x, x.flip(0))):
            want = V.quantise(want)[0]
            got = got.cpu().double()
            assert torch.equal(torch.isnan(got), torch.isnan(want)) and torch.equal(got.nan_to_num(), want.nan_to_num())


def test_8_bits_report_slots_past_the_pages():
    from block_diffusion_drafter_forward_gb300 import QuantKV, _lib
    status()
    kv = QuantKV(torch.zeros(2, 1, 32 * 64 + 32, dtype=torch.uint8, device="cuda"))
    x = torch.ones(3, 1, 64, device="cuda")
    kv.append(x, x, i32([32, 2 ** 31 - 1, 7]))
    assert status() == _lib.DFLASH_DEV_BAD_PAGE and status() == 0
    k, v = kv.read(i32([7, 32, 2 ** 31 - 1]), dtype=F32)
    assert status() == _lib.DFLASH_DEV_BAD_PAGE
    assert bool((k[0] == 1).all()) and bool((v[0] == 1).all()) and not k[1:].any() and not v[1:].any()
    assert [t.shape for t in kv.read(i32([]))] == [(0, 1, 64)] * 2
    kv.append(x[:0], x[:0], i32([]))


def cache8(ctx, new, nkv, hd, seed, gap=0):
    """Pages in 8 bits of sequences of ctx + new rows, by the library's own append; rows past each end all ones."""
    from block_diffusion_drafter_forward_gb300 import QuantKV
    lens = [c + n for c, n in zip(ctx, new)]
    pages = [-(-n // PAGE) for n in lens]
    total, mpps = sum(pages) + 2, max(pages) + 1
    g = torch.Generator(device="cuda").manual_seed(seed)
    perm = torch.randperm(total, generator=torch.Generator().manual_seed(seed)).to(torch.int32)
    table, at, slots = torch.full((len(ctx), mpps), -5, dtype=torch.int32), 0, []
    for s, n in enumerate(lens):
        table[s, :pages[s]] = perm[at:at + pages[s]]
        at += pages[s]
        j = torch.arange(n)
        slots.append(table[s].long()[j // PAGE] * PAGE + j % PAGE if n else j)
    kv = QuantKV(torch.full((total, nkv, 32 * hd + 32), 255, dtype=torch.uint8, device="cuda"))
    T = sum(lens)
    size = torch.ones(hd, device="cuda")
    size[5::32] = 10.0
    k = torch.randn(T, nkv, hd, generator=g, device="cuda") * size
    v = (torch.randn(T, nkv, hd, generator=g, device="cuda") + 0.3) * torch.exp2(torch.randint(-3, 4, (T, nkv, 1), generator=g, device="cuda").float())
    kv.append(k, v, torch.cat(slots).to(torch.int32).cuda())
    starts = [gap]
    for n in new:
        starts.append(starts[-1] + n)
    return kv, table.cuda(), lens, starts


ATTEND8 = [
    # ctx, new, nh, nkv, hd, window, causal, trees
    ([0], [1], 4, 1, 128, 0, True, False), ([4095], [1], 32, 4, 128, 0, True, False), ([15, 16, 17, 0], [1, 1, 1, 1], 8, 1, 64, 0, True, False),
    ([0], [33], 8, 1, 128, 0, True, False), ([5, 0, 100, 31], [3, 0, 17, 1], 16, 2, 128, 0, True, False),
    ([127, 128, 129, 255, 0], [1, 1, 1, 1, 1], 32, 4, 128, 0, True, False), ([300, 17], [16, 16], 32, 4, 128, 0, False, False),
    ([700, 40, 2100], [20, 300, 5], 64, 8, 128, 48, True, False), ([700, 40], [20, 129], 8, 1, 128, 1, True, False),
    ([50, 60], [40, 30], 8, 8, 64, 0, True, False), ([900, 3], [5, 70], 15, 3, 128, 0, True, False), ([900, 3], [1, 1], 14, 2, 64, 100, True, False),
    ([33], [40], 128, 1, 64, 0, True, False), ([1000, 16], [2, 1], 16, 2, 128, 0, True, False), ([1000, 16, 77], [2, 2, 2], 14, 2, 128, 0, False, False),
    ([6000, 0, 2500, 90], [1, 600, 3, 64], 32, 4, 128, 0, True, False), ([5000, 4000], [1, 1], 8, 1, 64, 1000, True, False),
    ([0], [1500], 16, 2, 128, 0, True, False), ([0], [1500], 16, 2, 64, 333, False, False),
    ([30000, 28001, 31977, 25000, 29999, 27000], [1] * 6, 32, 4, 128, 0, True, False),
    ([30000, 28001, 31977, 25000, 29999, 27000], [1, 1, 2, 1, 1, 3], 32, 4, 128, 0, True, False),
    ([20000, 28001, 21977], [1, 30, 2], 32, 4, 64, 0, True, False), ([300] * 200, [1] * 200, 16, 1, 128, 0, True, False),
    ([1, 2, 3, 4] * 90, [1] * 360, 8, 8, 64, 0, True, False), ([3000] * 40, [1, 40, 2, 1, 1, 300, 1, 17] * 5, 32, 4, 128, 0, True, False),
    ([4096], [32], 32, 4, 128, 0, True, True), ([127, 128, 129, 250, 16], [1, 16, 40, 63, 64], 32, 4, 128, 0, True, True),
    ([700, 40, 2100], [20, 200, 65], 64, 8, 128, 256, True, True), ([900, 3, 0], [1, 2, 2], 8, 1, 128, 64, True, True), ([6000, 0, 2500, 90], [33, 64, 1, 47], 16, 2, 64, 0, True, True),
    ([300, 0, 20], [2, 1, 2], 8, 1, 128, 0, True, True), ([100], [512], 8, 2, 128, 0, True, True),
]


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("trees", [24, 40])
def test_attend_many_trees(trees, kind):
    """Units of one and of two tiles, cut anywhere: trees of 1 to 100 nodes on contexts of up to 3000 rows."""
    from block_diffusion_drafter_forward_gb300 import PagedKV
    status()
    r = random.Random(trees)
    new = [r.choice([1, 16, 17, 32, 33, 47, 48, 49, 64, 100]) for _ in range(trees)]
    ctx = [r.randint(0, 3000) for _ in range(trees)]
    if kind == "e4m3":
        kv, table, lens, starts = cache8(ctx, new, 3, 128, trees)
        rows = lambda s, m: V.rows8(kv.pool, table[s], m)
    else:
        pool, table, lens, starts = cache(ctx, new, 3, 128, BF, trees)
        kv, rows = PagedKV(pool), V.rows16(pool, table)
    parents, plan = plan_of(new, lens, starts, trees)
    q = (torch.randn(starts[-1], 24, 128, generator=torch.Generator(device="cuda").manual_seed(trees), device="cuda") * 1.5).to(BF)
    out, lse = kv.attend(q, table, i32(lens), i32(starts), 100, tree=plan, lse=torch.empty(starts[-1], 24, device="cuda"))
    check_attend(out, lse, V.attend(q, rows, lens, starts, 1 / math.sqrt(128), parents=parents), slice(0, starts[-1]), 128)
    assert status() == 0


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("case", range(len(ATTEND8)))
def test_attend_in_8_bits(case, dtype):
    status()
    ctx, new, nh, nkv, hd, window, causal, trees = ATTEND8[case]
    kv, table, lens, starts = cache8(ctx, new, nkv, hd, case, gap=2)
    n = starts[-1] + 3
    parents, plan = plan_of(new, lens, starts, case, max(64, max(new))) if trees else (None, None)
    g = torch.Generator(device="cuda").manual_seed(case)
    wide = torch.randn(n, nh + 2, hd, generator=g, device="cuda").to(dtype)
    q = wide[:, 1:1 + nh]
    out, lse = torch.full((n, nh + 1, hd), 7.0, dtype=dtype, device="cuda"), torch.full((n, nh), 7.0, device="cuda")
    scale = 0.5 if case % 5 == 4 else 1 / math.sqrt(hd)
    if trees:
        plan = type(plan)(*(torch.cat([t, t[:3]]) for t in plan))
    kv.attend(q, table, i32(lens), i32(starts), max(new), causal=causal, window=window, scale=None if scale != 0.5 else 0.5,
              out=out[:, :nh], lse=lse, tree=plan)
    ref = V.attend(q, lambda s, m: V.rows8(kv.pool, table[s], m), lens, starts, scale, causal, window, parents)
    check_attend(out[:, :nh], lse, ref, slice(2, starts[-1]), hd)
    assert status() == 0
    untouched = torch.cat([out[:2], out[starts[-1]:]])
    assert bool((untouched == 7).all()) and bool((out[:, nh] == 7).all())
    assert bool((lse[:2] == 7).all()) and bool((lse[starts[-1]:] == 7).all())


@pytest.mark.parametrize("dtype", [BF, F32])
def test_attend_in_8_bits_rows_without_keys_and_out_of_range(dtype):
    from block_diffusion_drafter_forward_gb300 import _lib
    status()
    for new in ([20, 4], [1, 1]):
        kv, table, _, _ = cache8([0, 0], new, 2, 128, 3)
        lens, starts = [new[0] - 3 if new[0] > 3 else 0, 0], [0, new[0], sum(new)]
        q = torch.randn(sum(new), 16, 128, device="cuda").to(dtype)
        out, lse = kv.attend(q, table, i32(lens), i32(starts), max(new), lse=torch.empty(sum(new), 16, device="cuda"))
        ref = V.attend(q, lambda s, m: V.rows8(kv.pool, table[s], m), lens, starts, 1 / math.sqrt(128))
        check_attend(out, lse, ref, slice(0, sum(new)), 128)
        assert bool((out[new[0]:] == 0).all()) and bool((lse[new[0]:] == -math.inf).all()) and status() == 0
    for new in ([2, 3, 4], [1, 1, 1]):
        kv, table, lens, starts = cache8([40, 50, 60], new, 1, 128, 4)
        q = torch.randn(starts[-1], 8, 128, device="cuda").to(dtype)
        ref = V.attend(q, lambda s, m: V.rows8(kv.pool, table[s], m), lens, starts, 1 / math.sqrt(128))
        for bad in (-1, table.shape[1] * PAGE + 1):
            out = torch.full((starts[-1], 8, 128), 7.0, dtype=dtype, device="cuda")
            kv.attend(q, table, i32([lens[0], bad, lens[2]]), i32(starts), max(new), out=out)
            assert bool((out[starts[1]:starts[2]] == 7).all()) and status() == _lib.DFLASH_DEV_BAD_CTX
            check_attend(out, None, ref, slice(0, starts[1]), 128)
            check_attend(out, None, ref, slice(starts[2], starts[3]), 128)
        kv.attend(q, table, i32(lens), i32(starts[:3] + [starts[3] + 1]), max(new))
        assert status() == _lib.DFLASH_DEV_BAD_CTX
        broken = table.clone()
        broken[1, 1] = kv.pool.shape[0]
        kv.attend(q, broken, i32(lens), i32(starts), max(new))
        assert status() == _lib.DFLASH_DEV_BAD_PAGE


def test_attend_in_8_bits_over_all_powers():
    """Rows of very different sizes, beyond those whose power fits a single bf16 factor: V up to 2^110 and down to
    2^-100, K rows near zero and some of a few hundred."""
    from block_diffusion_drafter_forward_gb300 import QuantKV
    for n, hint in ((1, 1), (40, 40)):
        L = 400
        kv = QuantKV.empty(L // PAGE, 1, 128)
        g = torch.Generator(device="cuda").manual_seed(n)
        k = torch.randn(L, 1, 128, generator=g, device="cuda") * torch.exp2(torch.randint(-100, 3, (L, 1, 1), generator=g, device="cuda").float())
        v = torch.randn(L, 1, 128, generator=g, device="cuda") * torch.exp2(torch.randint(-100, 110, (L, 1, 1), generator=g, device="cuda").float())
        kv.append(k, v, torch.arange(L, dtype=torch.int32, device="cuda"))
        table = torch.arange(L // PAGE, dtype=torch.int32, device="cuda")[None]
        q = torch.randn(n, 8, 128, generator=g, device="cuda").to(BF)
        out, lse = kv.attend(q, table, i32([L]), i32([0, n]), hint, lse=torch.empty(n, 8, device="cuda"))
        check_attend(out, lse, V.attend(q, lambda s, m: V.rows8(kv.pool, table[s], m), [L], [0, n], 1 / math.sqrt(128)), slice(0, n), 128)
        # K of 2^20, one row: it takes all the weight, or none
        k[17] = 2.0 ** 20
        kv.append(k, v, torch.arange(L, dtype=torch.int32, device="cuda"))
        out, lse = kv.attend(q, table, i32([L]), i32([0, n]), hint, lse=torch.empty(n, 8, device="cuda"))
        check_attend(out, lse, V.attend(q, lambda s, m: V.rows8(kv.pool, table[s], m), [L], [0, n], 1 / math.sqrt(128)), slice(0, n), 128)


def test_attend_in_8_bits_in_a_graph_and_on_two_streams():
    """Captured once and replayed with other lengths and tables; and calls on two streams at once."""
    sides = [([3000, 20, 0, 511], [1, 1, 1, 1]), ([10, 800, 2000, 37], [1, 1, 1, 1]), ([3000, 20, 0, 511], [1, 16, 30, 2]), ([10, 800, 2000, 37], [16, 3, 1, 29])]
    for pair in (sides[:2], sides[2:]):
        states = [cache8(c, n, 4, 128, 11 + i) for i, (c, n) in enumerate(pair)]
        P, mp = max(s[0].pool.shape[0] for s in states), max(s[1].shape[1] for s in states)
        T, most = max(s[3][-1] for s in states), max(max(n) for _, n in pair)
        from block_diffusion_drafter_forward_gb300 import QuantKV
        kv = QuantKV.empty(P, 4, 128)
        table, lens, starts = torch.zeros(4, mp, dtype=torch.int32, device="cuda"), i32([0] * 4), i32([0] * 5)
        q = torch.randn(T, 32, 128, device="cuda").to(BF)
        out, lse = torch.zeros_like(q), torch.zeros(T, 32, device="cuda")

        def load(s):
            kv.pool[:s[0].pool.shape[0]].copy_(s[0].pool)
            table[:, :s[1].shape[1]].copy_(s[1])
            lens.copy_(i32(s[2]))
            starts.copy_(i32(s[3]))

        ref = [V.attend(q, lambda a, m: V.rows8(s[0].pool, s[1][a], m), s[2], s[3], 1 / math.sqrt(128)) for s in states]  # noqa: B023
        load(states[0])
        kv.attend(q, table, lens, starts, most, out=out, lse=lse)
        check_attend(out, lse, ref[0], slice(0, states[0][3][-1]), 128)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            kv.attend(q, table, lens, starts, most, out=out, lse=lse)
        for i in (1, 0, 1):
            load(states[i])
            out.zero_()
            graph.replay()
            check_attend(out, lse, ref[i], slice(0, states[i][3][-1]), 128)
        streams, outs = [torch.cuda.Stream() for _ in range(2)], [torch.zeros_like(q) for _ in range(2)]
        lens_of, starts_of = [i32(s[2]) for s in states], [i32(s[3]) for s in states]
        torch.cuda.synchronize()
        for _ in range(5):
            for i, st in enumerate(streams):
                states[i][0].attend(q, states[i][1], lens_of[i], starts_of[i], most, out=outs[i], stream=st)
        torch.cuda.synchronize()
        for i in range(2):
            check_attend(outs[i], None, ref[i], slice(0, states[i][3][-1]), 128)
    assert status() == 0


@pytest.mark.parametrize("new", [1, 40])
def test_pages_in_8_bits_past_32_bits(new):
    """Pages whose bytes lie beyond 2^32: written, read back and attended to."""
    from block_diffusion_drafter_forward_gb300 import QuantKV
    status()
    P = 2 ** 32 // (8 * 4128) + 40
    kv = QuantKV(torch.empty((P, 8, 4128), dtype=torch.uint8, device="cuda"))
    n = 100
    table = torch.arange(P - 1, P - 8, -1, dtype=torch.int32, device="cuda")[None].contiguous()
    j = torch.arange(n, device="cuda")
    slots = (table[0].long()[j // PAGE] * PAGE + j % PAGE).to(torch.int32)
    k, v = torch.randn(2, n, 8, 128, device="cuda").to(BF)
    kv.append(k, v, slots)
    for got, want in zip(kv.read(slots, dtype=F32), (k, v)):
        assert torch.equal(got.cpu().double(), V.quantise(want.cpu())[0])
    q = torch.randn(new, 32, 128, device="cuda").to(BF)
    out = kv.attend(q, table, i32([n]), i32([0, new]), new)
    ref = V.attend(q, lambda s, m: [V.quantise(x.cpu())[0] for x in (k, v)], [n], [0, new], 1 / math.sqrt(128))
    check_attend(out, None, ref, slice(0, new), 128)
    path = i32([[1] + list(range(3, 12))])
    kv.keep(table, i32([60]), path, i32([10]))
    for got, want in zip(kv.read(slots, dtype=F32), (k, v)):
        want = V.quantise(want.cpu())[0]
        want[60:70] = want[[61] + list(range(63, 72))]
        assert torch.equal(got.cpu().double(), want)
    assert status() == 0


# ------------------------------------------------------------------------------ together
@pytest.mark.parametrize("kind", ["bf16", "f32", "e4m3"])
def test_steps_of_verified_trees(kind):
    """Prompts, then steps that verify a tree per sequence and keep a branch of it: tables with pages held, tree
    plan, rotary positions, append, attention and the move, all on the device, against the dense
    computation over the branches that were kept, as if the other nodes had never been."""
    from block_diffusion_drafter_forward_gb300 import PagedKV, QuantKV, Rope, draft_tree, extend_tables
    status()
    nb, nkv, nh, hd, cap = 4, 2, 16, 128, 20
    dtype = F32 if kind == "f32" else BF
    g = torch.Generator(device="cuda").manual_seed(1)
    r = random.Random(3)
    kv = QuantKV.empty(nb * cap, nkv, hd) if kind == "e4m3" else PagedKV.empty(nb * cap, nkv, hd, dtype)
    kv.pool.fill_(255) if kind == "e4m3" else kv.pool.fill_(float("nan"))
    rope = Rope(64, 1e4)
    table, free, at, held = i32([[-1] * cap] * nb), torch.randperm(nb * cap, device="cuda").to(torch.int32), i32([0]), i32([0] * nb)
    ctx = [0] * nb
    past = [(torch.zeros(0, nkv, hd, dtype=torch.float64, device="cuda"),) * 2 for _ in range(nb)]
    for step, new in enumerate(([1, 70, 16, 33], [16, 30, 1, 40], [33, 1, 64, 20], [5, 17, 40, 64])):
        T = sum(new)
        plan = extend_tables(i32(ctx), i32(new), table, free, at, T + 3, held_pages=held)
        at = plan.free_end
        parents = [p for n in new for p in ([-1] + list(range(n - 1)) if step == 0 else some_tree(n, r.random()))]
        parents = parents + [0, 0, 0]
        tree = draft_tree(i32(parents), plan.kv_lens, plan.row_starts, 128)
        qkv = torch.randn(T + 3, (nh + 2 * nkv) * hd, generator=g, device="cuda").to(dtype)
        q, k, v = (x.view(T + 3, -1, hd) for x in qkv.split([nh * hd, nkv * hd, nkv * hd], 1))
        qr, kr = rope.rotate(q, tree.positions, k=k)
        kv.append(kr, v, plan.slots)
        out = kv.attend(qr, table, plan.kv_lens, plan.row_starts, max(new), tree=tree)
        assert bool((out[T:] == 0).all())
        i, paths = 0, []
        for s, n in enumerate(new):
            depth, see = V.tree(parents[i:i + n])
            assert tree.positions[i:i + n].tolist() == [ctx[s] + d for d in depth]
            fresh = [V.quantise(x[i:i + n].cpu())[0].cuda() if kind == "e4m3" else x[i:i + n].double() for x in (kr, v)]
            K, Vv = (torch.cat([a, b]).repeat_interleave(nh // nkv, 1) for a, b in zip(past[s], fresh))
            sc = torch.einsum("ihd,jhd->hij", qr[i:i + n].double(), K) / math.sqrt(hd)
            hide = torch.cat([torch.zeros(n, ctx[s], dtype=torch.bool), ~torch.tensor(see)], 1).cuda()
            p = torch.softmax(sc.masked_fill(hide, -math.inf), 2)
            want, spread = torch.einsum("hij,jhd->ihd", p, Vv), torch.einsum("hij,jhd->ihd", p, Vv.abs())
            half = torch.finfo(dtype).eps / 2
            # the output's rounding, P's where it is an operand in 16 bits, fp32 sums of scores of a few units
            assert bool(((out[i:i + n].double() - want).abs() <= half * want.abs() + (half + 2.0 ** -14) * spread).all())
            node, path = r.randrange(n) if step else n - 1, []
            while node >= 0:
                path.append(node)
                node = parents[i + node]
            paths.append(path[::-1])
            past[s] = tuple(torch.cat([a, b[paths[s]]]) for a, b in zip(past[s], fresh))
            i += n
        longest = max(map(len, paths))
        kv.keep(table, i32(ctx), i32([p + [0] * (longest - len(p)) for p in paths]), i32([len(p) for p in paths]))
        ctx = [c + len(p) for c, p in zip(ctx, paths)]
    assert status() == 0
