"""Trees, kept rows, pages in 8 bits and rotary positions without a GPU: what the C entries and the Python
calls refuse, the table of rotary frequencies, and the plain forms of the GPU tests by hand."""
import ctypes
import math
import os

import pytest
import torch

import verify_ref as V
from test_serve import pages


@pytest.fixture(scope="module")
def lib():
    from block_diffusion_drafter_forward_gb300 import _lib, build
    if not os.path.exists(_lib.LIB_PATH):
        build.build()
    return _lib.load()


def pages8(**kw):
    return pages(**{**dict(dtype=3, page_stride=2 * (32 * 128 + 32)), **kw})


def attend_args(**kw):
    a = dict(q_dtype=1, q=4096, q_stride=8 * 128, page_tables=4096, mpps=4, kv_lens=4096, row_starts=4096, nb=1, n_rows=1, max_new=1,
             nh=8, scale=1.0, window=0, causal=1, masks=4096, words=1, positions=4096, out=4096, out_stride=8 * 128, lse=None,
             workspace=None, workspace_bytes=0, stream=None)
    a.update(kw)
    return list(a.values())


BAD = [(dict(q_dtype=2), -1), (dict(q_dtype=3), -1), (dict(masks=None), -1), (dict(positions=None), -1), (dict(words=0), -1),
       (dict(words=9), -1), (dict(window=63), -5), (dict(window=127, words=2), -5), (dict(q=None), -1), (dict(nh=7), -1),
       (dict(q=4104), -1), (dict(nb=0), -1), (dict(nb=16385), -4), (dict(window=-1), -1), (dict(scale=math.nan), -1)]


@pytest.mark.parametrize("kw,code", BAD)
def test_attend_with_trees_refuses(lib, kw, code):
    for k in (pages(), pages8()):
        assert lib.dflash_attend_ex(ctypes.byref(k), *attend_args(**kw)) == code
        assert b"attend" in lib.dflash_last_error(None)


def test_attend_queries_have_the_pages_type(lib):
    assert lib.dflash_attend_ex(ctypes.byref(pages()), *attend_args(q_dtype=0)) == -1
    assert lib.dflash_attend_ex(ctypes.byref(pages(dtype=0)), *attend_args(q_dtype=1)) == -1
    for dt in (0, 1):
        assert lib.dflash_attend_ex(ctypes.byref(pages8()), *attend_args(q_dtype=dt, n_rows=0)) == 0
    assert lib.dflash_attend_ex(None, *attend_args()) == -1


@pytest.mark.parametrize("kw,code", [(dict(pool=None), -1), (dict(pool=4100), -1), (dict(dtype=2), -1), (dict(dtype=4), -1),
                                     (dict(head_dim=96), -5), (dict(n_kv_heads=0), -1), (dict(num_pages=0), -1), (dict(num_pages=1 << 27), -1),
                                     (dict(page_stride=2 * (32 * 128 + 32) - 16), -1), (dict(page_stride=2 * (32 * 128 + 32) + 8), -1)])
def test_pages_in_8_bits_are_checked(lib, kw, code):
    k = ctypes.byref(pages8(**kw))
    assert lib.dflash_append_kv_quant(k, 1, 4096, 256, 4096, 256, 4096, 1, None) == code
    assert lib.dflash_read_kv_quant(k, 1, 4096, 1, 4096, 256, 4096, 256, None) == code
    assert lib.dflash_keep_rows(k, 4096, 4, 4096, 1, 4096, 4, 4096, None) == code
    assert lib.dflash_attend_ex(k, *attend_args()) == code
    assert lib.dflash_attend_workspace(k) == code


def test_attend_over_8_bits_without_the_queries_type(lib):
    import test_serve
    assert lib.dflash_attend(ctypes.byref(pages8()), *test_serve.attend_args(n_rows=0)) == 0
    assert lib.dflash_attend(ctypes.byref(pages8()), *test_serve.attend_args(q=None)) == -1
    assert lib.dflash_attend(ctypes.byref(pages8()), *test_serve.attend_args(q_stride=1028)) == -1


def test_calls_for_other_pages_refuse_those_in_8_bits(lib):
    k = ctypes.byref(pages8())
    assert lib.dflash_append_kv(k, 4096, 256, 4096, 256, 4096, 1, None) == -1
    for f in (pages(), pages(dtype=0)):
        assert lib.dflash_append_kv_quant(ctypes.byref(f), 1, 4096, 256, 4096, 256, 4096, 1, None) == -1
        assert lib.dflash_read_kv_quant(ctypes.byref(f), 1, 4096, 1, 4096, 256, 4096, 256, None) == -1
        assert b"e4m3" in lib.dflash_last_error(None)


@pytest.mark.parametrize("dt,k,ks,v,vs,slots,n,code", [
    (2, 4096, 256, 4096, 256, 4096, 1, -1), (3, 4096, 256, 4096, 256, 4096, 1, -1), (1, None, 256, 4096, 256, 4096, 1, -1),
    (1, 4096, 256, None, 256, 4096, 1, -1), (1, 4096, 256, 4096, 256, None, 1, -1), (1, 4096, 256, 4096, 256, 4096, -1, -1),
    (1, 4096, 248, 4096, 256, 4096, 1, -1), (1, 4096, 256, 4096, 260, 4096, 1, -1), (0, 4096, 256, 4096, 258, 4096, 1, -1),
    (1, 4098, 256, 4096, 256, 4096, 1, -1), (0, 4096, 256, 4104, 256, 4096, 1, -1), (1, None, 0, None, 0, None, 0, 0)])
def test_rows_in_and_out_of_8_bits_refuse(lib, dt, k, ks, v, vs, slots, n, code):
    p = ctypes.byref(pages8())
    assert lib.dflash_append_kv_quant(p, dt, k, ks, v, vs, slots, n, None) == code
    assert lib.dflash_read_kv_quant(p, dt, slots, n, k, ks, v, vs, None) == code


def tree_args(**kw):
    a = dict(parents=4096, kv=4096, rs=4096, nb=1, n=1, most=64, pos=4096, masks=4096, status=None, stream=None)
    a.update(kw)
    return list(a.values())


@pytest.mark.parametrize("kw,code", [(dict([(n, None)]), -1) for n in ("parents", "kv", "rs", "pos", "masks")] +
                         [(dict(nb=0), -1), (dict(n=-1), -1), (dict(nb=16385), -4), (dict(n=(1 << 30) + 1), -4), (dict(most=0), -5),
                          (dict(most=513), -5), (dict(n=0), 0)])
def test_trees_refuse(lib, kw, code):
    assert lib.dflash_draft_tree(*tree_args(**kw)) == code
    assert code == 0 or b"draft_tree" in lib.dflash_last_error(None)


@pytest.mark.parametrize("args,code", [((None, 4, 4096, 1, 4096, 4, 4096), -1), ((4096, 4, None, 1, 4096, 4, 4096), -1),
                                       ((4096, 4, 4096, 1, None, 4, 4096), -1), ((4096, 4, 4096, 1, 4096, 4, None), -1),
                                       ((4096, 0, 4096, 1, 4096, 4, 4096), -1), ((4096, 1 << 26, 4096, 1, 4096, 4, 4096), -1),
                                       ((4096, 4, 4096, 0, 4096, 4, 4096), -1), ((4096, 4, 4096, 1, 4096, -1, 4096), -1),
                                       ((4096, 4, 4096, 16385, 4096, 4, 4096), -4), ((4096, 4, 4096, 1, 4096, 513, 4096), -4)])
def test_keep_refuses(lib, args, code):
    for k in (pages(), pages8(), pages(dtype=0)):
        assert lib.dflash_keep_rows(ctypes.byref(k), *args, None) == code
        assert b"keep_rows" in lib.dflash_last_error(None)


def rotate_args(**kw):
    a = dict(q=4096, qs=8 * 128, qo=8192, qos=8 * 128, qh=8, k=4096, ks=256, ko=8192, kos=256, kh=2, dtype=1, rows=1, hd=128, rd=128,
             inter=0, inverse=0, pos=4096, turns=4096, mscale=1.0, stream=None)
    a.update(kw)
    return list(a.values())


@pytest.mark.parametrize("kw,code", [
    (dict(q=None), -1), (dict(qo=None), -1), (dict(k=None), -1), (dict(ko=None), -1), (dict(pos=None), -1), (dict(turns=None), -1),
    (dict(dtype=2), -1), (dict(rows=-1), -1), (dict(rows=(1 << 30) + 1), -4), (dict(hd=120), -5), (dict(hd=528), -5), (dict(hd=0), -5),
    (dict(rd=8), -5), (dict(rd=24), -5), (dict(rd=144), -5), (dict(qh=0), -1), (dict(kh=-1), -1), (dict(qh=4095), -1), (dict(qs=1020), -1),
    (dict(qs=1028), -1), (dict(kos=248), -1), (dict(q=4104), -1), (dict(ko=4100), -1), (dict(mscale=math.inf), -1), (dict(mscale=math.nan), -1),
    (dict(qo=4096, qos=2048), -1), (dict(ko=4096, kos=512), -1), (dict(qs=1 << 62), -1), (dict(rows=0, q=None), 0)])
def test_rotate_refuses(lib, kw, code):
    assert lib.dflash_rotate(*rotate_args(**kw)) == code
    assert code == 0 or b"rotate" in lib.dflash_last_error(None)


YARN = (32.0, 8192.0, 32.0, 1.0)


@pytest.mark.parametrize("rd,theta,linear,yarn", [(128, 1e6, 1.0, None), (64, 1e4, 4.0, None), (16, 5e5, 1.0, None), (128, 1e6, 1.0, YARN),
                                                  (48, 1e4, 1.0, YARN), (512, 2.0, 1.0, None), (64, 1e4, 1.0, (4.0, 32.0, 32.0, 32.0))])
def test_rope_table(lib, rd, theta, linear, yarn):
    from block_diffusion_drafter_forward_gb300 import dflash_rope_turns
    turns, mscale = dflash_rope_turns(rd, theta, linear, yarn)
    want, scale = V.inv_freq(rd, theta, linear, yarn)
    assert len(turns) == rd // 2 and mscale == pytest.approx(scale, rel=2.0 ** -23)
    for t, f in zip(turns, want):  # a few roundings of 2^-53, the power's among them, and the last unit
        assert abs(t - f / (2 * math.pi) * 2.0 ** 64) <= t * 2.0 ** -48 + 1
    assert max(turns) < 2 ** 62


@pytest.mark.parametrize("args", [(24, 1e4), (8, 1e4), (528, 1e4), (64, 1.0), (64, math.inf), (64, 1e4, 0.5), (64, 1e4, math.nan), (64, 1e4, 2.0, YARN),
                                  (64, 1e4, 1.0, (0.5, 1.0, 1.0, 1.0)), (64, 1e4, 1.0, (2.0, 0.0, 1.0, 1.0)), (64, 1e4, 1.0, (2.0, 8.0, -1.0, 1.0))])
def test_rope_table_refuses(lib, args):
    from block_diffusion_drafter_forward_gb300 import DflashError, dflash_rope_turns
    with pytest.raises(DflashError, match="rope_turns"):
        dflash_rope_turns(*args)


def test_rope_table_refuses_null(lib):
    f = ctypes.c_float()
    assert lib.dflash_rope_turns(64, 1e4, 1.0, 0, 1.0, 1.0, 1.0, 1.0, None, ctypes.byref(f)) == -1
    assert lib.dflash_rope_turns(64, 1e4, 1.0, 0, 1.0, 1.0, 1.0, 1.0, (ctypes.c_uint64 * 32)(), None) == -1


def test_python_calls_refuse_host_tensors():
    from block_diffusion_drafter_forward_gb300 import QuantKV, Rope, draft_tree
    z = torch.zeros(4, dtype=torch.int32)
    with pytest.raises(ValueError, match="parents: expected a cuda tensor"):
        draft_tree(z, z, z, 4)
    with pytest.raises(ValueError, match="pool: expected a cuda tensor"):
        QuantKV(torch.zeros(2, 1, 32 * 64 + 32, dtype=torch.uint8))
    rope = Rope(64, 1e4, device="cpu")
    with pytest.raises(ValueError, match="q: expected a cuda tensor"):
        rope.rotate(torch.zeros(1, 1, 64), z[:1])
    with pytest.raises(TypeError, match="q: expected"):
        rope.rotate([1.0], z[:1])


# ------------------------------------------------------------------------------ plain forms by hand
def test_plain_tree_by_hand():
    depth, see = V.tree([-1, 0, 0, 1, -1, 3])
    assert depth == [0, 1, 1, 2, 0, 3]
    assert [[j for j in range(6) if r[j]] for r in see] == [[0], [0, 1], [0, 2], [0, 1, 3], [4], [0, 1, 3, 5]]
    assert V.words(see, 1) == [[1], [3], [5], [11], [16], [43]]
    deep = V.words(V.tree([-1] + list(range(69)))[1], 2)
    assert deep[63] == [-1, 0] and deep[69] == [-1, 63]


def test_plain_codes_by_hand():
    """Every e4m3 value is its own nearest; halves between neighbours go to the even one; the row's power."""
    vals = sorted({V.code_value(c) for c in range(256) if c & 127 != 127})
    x = torch.tensor(vals + [0.0] * (256 - len(vals)), dtype=torch.float64)
    y, e = V.quantise(x[None])
    assert int(e) == 127 and torch.equal(y[0], x)
    mid = (x[:252] + x[1:253]) / 2
    y, _ = V.quantise(torch.cat([mid, x[-1:], torch.tensor([448.0])])[None])
    near = torch.minimum((y[0, :252] - x[:252]).abs(), (y[0, :252] - x[1:253]).abs())
    assert bool((near == 0).all())
    codes = {v: c for c in range(256) if c & 127 != 127 for v in [V.code_value(c)]}
    assert all(codes[v] % 2 == 0 for v in y[0, :252].tolist())
    for top, k in ((448.0, 0), (448.5, 1), (224.0, -1), (224.5, 0), (1.0, -8), (2.0 ** -200, -118), (3e38, 119), (0.0, -118)):
        assert int(V.quantise(torch.tensor([[top, 0.0]]).double())[1]) == k + 127
    y, e = V.quantise(torch.tensor([[math.inf, 1.0, math.nan, -math.inf]]).double())
    assert int(e) == 119 and y[0, 1] == 1 and bool(torch.isnan(y[0, [0, 2, 3]]).all())


def test_plain_pages_are_inverse():
    g = torch.Generator().manual_seed(0)
    for hd in (64, 128):
        for off in (V.k8, V.v8):
            assert sorted(off(j, d) for j in range(16) for d in range(hd)) == list(range(16 * hd))
        k, v = torch.randn(20, 2, hd, generator=g), torch.randn(20, 2, hd, generator=g) * 100
        table = torch.tensor([2, 0], dtype=torch.int32)
        pool = V.put8(torch.zeros(3, 2, 32 * hd + 32, dtype=torch.uint8), k, v, [int(table[i // 16]) * 16 + i % 16 for i in range(20)])
        kk, vv = V.rows8(pool, table, 20)
        assert torch.equal(kk, V.quantise(k)[0]) and torch.equal(vv, V.quantise(v)[0])
        # half a step of e4m3 relative to the value, or half the smallest step of the row
        for a, b in ((kk, k), (vv, v)):
            unit = b.double().abs().amax(-1, keepdim=True) / 224
            assert bool(((a - b.double()).abs() <= torch.maximum(2.0 ** -4 * b.double().abs(), 2.0 ** -10 * unit)).all())


def test_plain_rotate_by_hand():
    x = torch.tensor([[[1.0, 2.0, 3.0, 4.0, 9.0]]], dtype=torch.float64)
    quarter = [2 ** 62, 0]  # a quarter turn per position, none
    one = torch.tensor([1])
    assert torch.allclose(V.rotate(x, one, quarter, 1.0, False)[0], torch.tensor([-3.0, 2, 1, 4, 9]).double())
    assert torch.allclose(V.rotate(x, one, quarter, 1.0, True)[0], torch.tensor([-2.0, 1, 3, 4, 9]).double())
    assert torch.allclose(V.rotate(x, torch.tensor([-1]), quarter, 2.0, False)[0], torch.tensor([6.0, 4, -2, 8, 9]).double())
    back = V.rotate(V.rotate(x, one * 7, [2 ** 61, 12345678901234567], 1.0, True)[0], one * 7, [2 ** 61, 12345678901234567], 1.0, True, True)[0]
    assert torch.allclose(back, x)
