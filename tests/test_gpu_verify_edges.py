"""Calls at the edges of trees, kept rows, rotary positions and pages in 8 bits: NaN that a cache holds, sizes past its
tables, tables of the caller's own."""
import math

import pytest
import torch

import verify_ref as V
from test_gpu_serve import cache, check_attend
from test_gpu_verify import cache8, i32, plan_of, status

pytestmark = pytest.mark.gpu
PAGE = 16
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


# ------------------------------------------------------------------------------ NaN in pages of 8 bits
def sees(lens, starts, causal, window, parents):
    """[rows, longest] truth values: which keys of its sequence a row sees."""
    out = torch.zeros(starts[-1], max(lens), dtype=torch.bool)
    for s, kv in enumerate(lens):
        n = starts[s + 1] - starts[s]
        ctx = kv - n
        own = V.tree(parents[starts[s]:starts[s + 1]]) if parents else None
        for i in range(n):
            pos = ctx + (own[0][i] if parents else i)
            row = out[starts[s] + i]
            row[:kv] = True
            if window:
                row[:max(0, pos - window + 1)] = False
            if parents:
                row[ctx:kv] = torch.tensor(own[1][i])
            elif causal:
                row[pos + 1:] = False
    return out


NANS = [
    # ctx, new, nh, nkv, hd, window, causal, trees
    ([37], [1], 8, 1, 128, 0, True, False), ([3000, 100], [1, 1], 32, 4, 128, 0, True, False), ([500, 90], [2, 2], 16, 2, 64, 40, True, False),
    ([600, 17], [16, 5], 16, 2, 128, 0, True, False), ([2000, 0], [16, 40], 32, 4, 64, 100, True, False), ([300, 50], [16, 9], 8, 1, 128, 0, False, False),
    ([700, 200, 0, 40] * 10, [17, 64, 20, 33] * 10, 32, 4, 128, 0, True, False), ([400, 900] * 12, [40, 30] * 12, 16, 4, 64, 64, True, False),
    ([0], [1500], 16, 2, 128, 0, True, False), ([100, 30], [2, 1], 8, 1, 128, 0, True, True), ([2500, 60], [32, 7], 16, 2, 128, 0, True, True),
    ([700, 200, 0, 40] * 8, [33, 64, 20, 50] * 8, 32, 4, 128, 128, True, True), ([300] * 24, [40, 17] * 12, 16, 4, 64, 0, True, True),
]


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("case", range(len(NANS)))
def test_nan_in_8_bits_reaches_the_rows_that_see_it(case, dtype):
    """NaN in K (the whole row of the output) and in V (its dim), of the context and of rows that others hide: every row that
    sees one has it, and the others have the numbers that they would have had."""
    status()
    ctx, new, nh, nkv, hd, window, causal, trees = NANS[case]
    kv, table, lens, starts = cache8(ctx, new, nkv, hd, case)
    parents, plan = plan_of(new, lens, starts, case, max(64, max(new))) if trees else (None, None)
    n = starts[-1]
    g = torch.Generator(device="cuda").manual_seed(case)
    q = torch.randn(n, nh, hd, generator=g, device="cuda").to(dtype)
    # of every second sequence: in V a context row and three of its last ones, by either sign's code, and in K its last row
    pool, bad_k, bad_v = kv.pool, {}, {}
    for s in range(0, len(lens), 2):
        L = lens[s]
        at = {j for j in (L * 2 // 3, L - 1, L - new[s] // 2 - 1, L - new[s]) if 0 <= j < L}
        for x, j in enumerate(sorted(at)):
            page, h, d = int(table[s, j // PAGE]), (x + s) % nkv, (7 * x + 31 * s + 5) % hd
            pool[page, h, 16 * hd + V.v8(j % PAGE, d)] = 127 if x % 2 else 255
            bad_v.setdefault((s, h), []).append((j, d))
        if s % 4 == 0 and case % 3:
            j, h = L - 1, (s // 4) % nkv
            pool[int(table[s, j // PAGE]), h, V.k8(j % PAGE, (3 * s + 11) % hd)] = 255 if s % 8 else 127
            bad_k.setdefault((s, h), []).append(j)
    rows = lambda s, m: [x.nan_to_num() for x in V.rows8(pool, table[s], m)]
    scale = 1 / math.sqrt(hd)
    out, lse, spread, dots = V.attend(q, rows, lens, starts, scale, causal, window, parents)
    see = sees(lens, starts, causal, window, parents).cuda()
    group = nh // nkv
    for (s, h), at in bad_v.items():
        for j, d in at:
            r = starts[s] + see[starts[s]:starts[s + 1], j].nonzero()[:, 0]
            out[r[:, None], torch.arange(h * group, h * group + group, device="cuda")[None], d] = math.nan
    for (s, h), at in bad_k.items():
        for j in at:
            r = (starts[s] + see[starts[s]:starts[s + 1], j].nonzero()[:, 0])[:, None]
            heads = torch.arange(h * group, h * group + group, device="cuda")[None]
            out[r, heads], lse[r, heads] = math.nan, math.nan
    assert bool(torch.isnan(out).any()) and not bool(torch.isnan(out).all())
    got, got_lse = kv.attend(q, table, i32(lens), i32(starts), max(new), causal=causal, window=window, tree=plan,
                             lse=torch.empty(n, nh, device="cuda"))
    assert torch.equal(torch.isnan(got), torch.isnan(out)) and torch.equal(torch.isnan(got_lse), torch.isnan(lse))
    gone, whole = torch.isnan(out), torch.isnan(lse)
    check_attend(got.masked_fill(gone, 0), got_lse.masked_fill(whole, 0),
                 (out.masked_fill(gone, 0), lse.masked_fill(whole, 0), spread, dots), slice(0, n), hd)
    assert status() == 0


def test_a_slot_named_twice_in_8_bits_spoils_no_other():
    """Singles and runs of eight aimed at one slot: what that slot holds is open, the others' bytes are not."""
    from block_diffusion_drafter_forward_gb300 import QuantKV
    status()
    g = torch.Generator().manual_seed(1)
    slots = list(range(40)) + [5, 5, 39, -1, 47] + list(range(16, 24))
    twice = {5, 39} | set(range(16, 24))
    k, v = torch.randn(2, len(slots), 2, 64, generator=g)
    kv = QuantKV(torch.zeros(3, 2, 32 * 64 + 32, dtype=torch.uint8, device="cuda"))
    kv.append(k.cuda(), v.cuda(), i32(slots))
    got = kv.read(i32(list(range(48))), dtype=F32)
    for x, y in zip(got, (k, v)):
        for j in range(48):
            if j not in twice:
                want = V.quantise(y[slots.index(j)])[0] if j in slots else torch.zeros(2, 64).double()
                assert torch.equal(x[j].cpu().double(), want), j
    assert status() == 0


# ------------------------------------------------------------------------------ kept rows
@pytest.mark.parametrize("kind", ["bf16", "f32", "e4m3"])
def test_keep_reports_contexts_past_the_table(kind):
    """Also where no row is kept, up to the largest numbers: the pages stay as they are, and the call ends."""
    from block_diffusion_drafter_forward_gb300 import PagedKV, QuantKV, _lib
    status()
    kv = QuantKV.empty(8, 3, 64) if kind == "e4m3" else PagedKV.empty(8, 3, 64, BF if kind == "bf16" else F32)
    kv.pool.random_(0, 100)
    before = kv.pool.clone()
    table, path = i32([[0, 1, 2]]), i32([[0, 2]])
    for ctx, n, want in ((48, 0, 0), (47, 0, 0), (0, 0, 0), (46, 1, 0), (49, 0, _lib.DFLASH_DEV_BAD_CTX), (61, 0, _lib.DFLASH_DEV_BAD_CTX),
                         (1000, 0, _lib.DFLASH_DEV_BAD_CTX), (-1, 0, _lib.DFLASH_DEV_BAD_CTX), (47, 2, _lib.DFLASH_DEV_BAD_CTX),
                         (48, 1, _lib.DFLASH_DEV_BAD_CTX), (2 ** 31 - 31, 0, _lib.DFLASH_DEV_BAD_CTX), (2 ** 31 - 1, 0, _lib.DFLASH_DEV_BAD_CTX),
                         (2 ** 31 - 1, 2, _lib.DFLASH_DEV_BAD_CTX), (-2 ** 31, 1, _lib.DFLASH_DEV_BAD_CTX)):
        kv.keep(table, i32([ctx]), path, i32([n]))
        assert status() == want and torch.equal(kv.pool, before), (ctx, n)


# ------------------------------------------------------------------------------ rotary positions
@pytest.mark.parametrize("inter", [False, True])
def test_sines_and_cosines_in_32_bits(inter):
    """Of (1, 0) a rotation leaves (cos, sin) without another rounding: what is left of the angle, at most an eighth of a turn,
    in fp32 half turns below 1/4 (2^-27, pi of which are 0.4 2^-24), its cut at 2^-32 turns (0.03 2^-24) and the last place that
    sine and cosine may be off by (2^-24 below 1)."""
    from block_diffusion_drafter_forward_gb300 import Rope
    for theta, far in ((1e4, 2 ** 31 - 1), (1e6, 100000), (10.0, 2 ** 31 - 1)):
        rope = Rope(128, theta, interleaved=inter)
        pos = torch.randint(-far, far, (3000,), generator=torch.Generator().manual_seed(int(theta)))
        pos[:9] = torch.tensor([0, 1, -1, 2 ** 31 - 1, -2 ** 31, 2, 3, 4, 5])
        x = torch.zeros(3000, 1, 128, device="cuda")
        x[..., 0::2] = 1.0 if inter else 0.0
        x[..., :64] += 0.0 if inter else 1.0
        for inverse in (False, True):
            want, _ = V.rotate(x.double(), pos, rope.turns.tolist(), 1.0, inter, inverse)
            got = rope.rotate(x, i32(pos.tolist()), inverse=inverse)
            assert float((got.double() - want).abs().max()) <= 1.43 * 2.0 ** -24


def test_rotate_with_a_table_of_the_callers_own():
    from block_diffusion_drafter_forward_gb300 import Rope
    rope = Rope(64, 1e4)
    q, pos = torch.randn(50, 2, 64, device="cuda"), torch.arange(50, dtype=torch.int32, device="cuda") * 1000
    table = [(j * 0x123456789ABCDEF + 2 ** 40) % 2 ** 62 for j in range(32)]
    for scale in (1.0, 1.5):
        table.reverse()
        rope.turns, rope.mscale = torch.tensor(table, dtype=torch.int64, device="cuda"), scale
        torch.empty(32, dtype=torch.int64, device="cuda").fill_(0)  # takes the place of the table before, if that is free
        want, size = V.rotate(q.double(), pos.cpu(), table, scale, False)
        # sine and cosine to 1.43 2^-24, the scale, two products and their sum to 2^-24 each, the result
        assert bool(((rope.rotate(q, pos).double() - want).abs() <= 5 * 2.0 ** -24 * size).all())
    kept = rope.turns
    for bad in (kept[:31], kept.int(), torch.zeros(64, dtype=torch.int64, device="cuda")[::2]):
        with pytest.raises(ValueError, match="turns"):
            rope.turns = bad
    with pytest.raises(TypeError, match="turns"):
        rope.turns = table
    assert rope.turns is kept
    rope.turns = kept.cpu()
    with pytest.raises(ValueError, match="the table is on cpu"):
        rope.rotate(q, pos)
    rope.turns = kept.clone()
    rope.turns.resize_(31)
    with pytest.raises(ValueError, match="turns"):
        rope.rotate(q, pos)


# ------------------------------------------------------------------------------ chains
@pytest.mark.parametrize("kind", ["bf16", "f32", "e4m3"])
def test_a_chain_against_the_causal_form_in_64_bits(kind):
    """A tree that is one chain, by any hint: within the roundings of a causal chunk, lse included (a key hidden or seen beside
    the right ones is off by more)."""
    from block_diffusion_drafter_forward_gb300 import PagedKV, draft_tree
    status()
    ctx, new = [333, 20, 1000, 0], [16, 1, 64, 130]
    if kind == "e4m3":
        kv, table, lens, starts = cache8(ctx, new, 2, 128, 5)
        rows = lambda s, m: V.rows8(kv.pool, table[s], m)
    else:
        pool, table, lens, starts = cache(ctx, new, 2, 128, BF if kind == "bf16" else F32, 5)
        kv, rows = PagedKV(pool), V.rows16(pool, table)
    plan = draft_tree(i32([p for n in new for p in [-1] + list(range(n - 1))]), i32(lens), i32(starts), 300)
    n = starts[-1]
    g = torch.Generator(device="cuda").manual_seed(3)
    for dtype in ((BF, F32) if kind == "e4m3" else (kv.pool.dtype,)):
        q = torch.randn(n, 16, 128, generator=g, device="cuda").to(dtype)
        ref = V.attend(q, rows, lens, starts, 1 / math.sqrt(128))
        for hint in (0, 64, 500):
            for tree in (plan, None):
                out, lse = kv.attend(q, table, i32(lens), i32(starts), hint, tree=tree, lse=torch.empty(n, 16, device="cuda"))
                check_attend(out, lse, ref, slice(0, n), 128)
    assert status() == 0


# ------------------------------------------------------------------------------ the C entries by their names
def test_entries_by_their_names_are_the_calls():
    """Each entry called with addresses does what the tensor call of it does, to the last bit."""
    import block_diffusion_drafter_forward_gb300 as D
    status()
    g = torch.Generator(device="cuda").manual_seed(7)
    nb, nodes, nh, nkv, hd, ctx = 3, 5, 16, 2, 128, (30, 0, 77)
    parents = i32([-1, 0, 0, 1, -1] * nb)
    lens, starts, table = i32([c + nodes for c in ctx]), i32([0, 5, 10, 15]), torch.arange(18, dtype=torch.int32, device="cuda").view(3, 6)
    plan = D.draft_tree(parents, lens, starts, nodes)
    pos, masks = torch.empty_like(plan.positions), torch.empty_like(plan.masks)
    D.dflash_draft_tree(parents.data_ptr(), lens.data_ptr(), starts.data_ptr(), nb, 15, nodes, pos.data_ptr(), masks.data_ptr())
    assert torch.equal(pos, plan.positions) and torch.equal(masks, plan.masks)

    rope = D.Rope(64, 1e4)
    q, k = torch.randn(15, nh, hd, generator=g, device="cuda").to(BF), torch.randn(15, nkv, hd, generator=g, device="cuda").to(BF)
    want = rope.rotate(q, pos, k=k, inverse=True)
    qo, ko = torch.empty_like(q), torch.empty_like(k)
    D.dflash_rotate(q.data_ptr(), nh * hd, qo.data_ptr(), nh * hd, nh, k.data_ptr(), nkv * hd, ko.data_ptr(), nkv * hd, nkv, 1, 15, hd, 64, 0, 1,
                    pos.data_ptr(), rope.turns.data_ptr(), rope.mscale)
    assert torch.equal(qo, want[0]) and torch.equal(ko, want[1])

    L = int(lens.sum())
    rows = torch.randn(2, L, nkv, hd, generator=g, device="cuda").to(BF)
    slots = i32([s * 96 + j for s, n in enumerate(lens.tolist()) for j in range(n)])
    a, b = D.QuantKV(torch.zeros(18, nkv, 32 * hd + 32, dtype=torch.uint8, device="cuda")), D.QuantKV(torch.zeros(18, nkv, 32 * hd + 32, dtype=torch.uint8, device="cuda"))
    a.append(*rows, slots)
    D.dflash_append_kv_quant(b._c, 1, rows[0].data_ptr(), nkv * hd, rows[1].data_ptr(), nkv * hd, slots.data_ptr(), L)
    assert torch.equal(a.pool, b.pool) and bool(a.pool.any())
    back = torch.empty(2, L, nkv, hd, device="cuda")
    D.dflash_read_kv_quant(b._c, 0, slots.data_ptr(), L, back[0].data_ptr(), nkv * hd, back[1].data_ptr(), nkv * hd)
    for x, y in zip(a.read(slots, dtype=F32), back):
        assert torch.equal(x, y)

    c = D.PagedKV(torch.zeros(18, nkv, 2, 16 * hd, dtype=BF, device="cuda"))
    c.append(*rows, slots)
    for kv in (a, c):
        need = D.dflash_attend_workspace(kv._c)
        ws, scale = torch.empty(need, dtype=torch.uint8, device="cuda"), 1 / math.sqrt(hd)
        for tree in (plan, None):
            out, lse = torch.zeros(15, nh, hd, dtype=BF, device="cuda"), torch.empty(15, nh, device="cuda")
            D.dflash_attend_ex(kv._c, 1, q.data_ptr(), nh * hd, table.data_ptr(), 6, lens.data_ptr(), starts.data_ptr(), nb, 15, nodes, nh, scale, 0, 1,
                               masks.data_ptr() if tree else 0, 1 if tree else 0, pos.data_ptr() if tree else 0, out.data_ptr(), nh * hd,
                               lse.data_ptr(), ws.data_ptr(), need)
            y, l = kv.attend(q, table, lens, starts, nodes, tree=tree, lse=torch.empty(15, nh, device="cuda"))
            assert torch.equal(out, y) and torch.equal(lse, l) and bool(y.any())
        D.dflash_attend(kv._c, q.data_ptr(), nh * hd, table.data_ptr(), 6, lens.data_ptr(), starts.data_ptr(), nb, 15, nodes, nh, scale, 0, 1,
                        out.zero_().data_ptr(), nh * hd, lse.data_ptr(), ws.data_ptr(), need)
        assert torch.equal(out, y) and torch.equal(lse, l)
        path, n_path, at = i32([[0, 1, 3], [0, 2, 9], [4, 9, 9]]), i32([3, 2, 1]), i32(list(ctx))
        twin = type(kv)(kv.pool.clone())
        kv.keep(table, at, path, n_path)
        D.dflash_keep_rows(twin._c, table.data_ptr(), 6, at.data_ptr(), nb, path.data_ptr(), 3, n_path.data_ptr())
        assert torch.equal(kv.pool, twin.pool)
    assert status() == 0


# ------------------------------------------------------------------------------ hints
@pytest.mark.parametrize("nb", [1, 40])
def test_single_token_form_with_chunks_of_many_tiles(nb):
    """A hint of one token for sequences of which some have hundreds: the units of 16 rows all the same, with a NaN among the
    keys of one too."""
    status()
    new = ([700] if nb == 1 else [600] + [1, 2] * 10 + [900] + [1] * 18)
    ctx = [(37 * i) % 300 for i in range(len(new))]
    kv, table, lens, starts = cache8(ctx, new, 2, 64, nb)
    n = starts[-1]
    q = torch.randn(n, 16, 64, generator=torch.Generator(device="cuda").manual_seed(nb), device="cuda").to(BF)
    ref = V.attend(q, lambda s, m: V.rows8(kv.pool, table[s], m), lens, starts, 1 / 8)
    rows = i32(lens), i32(starts)
    out, lse = kv.attend(q, table, *rows, 1, lse=torch.empty(n, 16, device="cuda"))
    check_attend(out, lse, ref, slice(0, n), 64)
    j, d = lens[0] - 300, 33                                     # rows 400 on of the first sequence see it, by the first K/V head
    kv.pool[int(table[0, j // PAGE]), 0, 16 * 64 + V.v8(j % PAGE, d)] = 127
    got, again = kv.attend(q, table, *rows, 1, lse=torch.empty(n, 16, device="cuda"))
    gone = torch.zeros_like(got, dtype=torch.bool)
    gone[new[0] - 300:new[0], :8, d] = True
    assert torch.equal(torch.isnan(got), gone) and torch.equal(got[~gone], out[~gone]) and torch.equal(again, lse)
    assert status() == 0
