"""The serving operators without a GPU: what the C entries and the Python calls refuse, the struct's
layout, and the plain forms of the GPU tests against small cases worked out by hand."""
import ctypes
import os

import numpy as np
import pytest
import torch

import serve_ref as R


@pytest.fixture(scope="module")
def lib():
    from block_diffusion_drafter_forward_gb300 import _lib, build
    if not os.path.exists(_lib.LIB_PATH):
        build.build()
    return _lib.load()


def pages(**kw):
    from block_diffusion_drafter_forward_gb300 import _lib
    k = _lib.dflash_kv_pages()
    d = dict(pool=4096, page_stride=32 * 2 * 128, status=None, dtype=_lib.DFLASH_BF16, n_kv_heads=2, head_dim=128, num_pages=8)
    d.update(kw)
    for f, v in d.items():
        setattr(k, f, v)
    return k


BAD_PAGES = [(dict(pool=None), -1), (dict(pool=4100), -1), (dict(dtype=2), -1), (dict(head_dim=96), -5),
             (dict(n_kv_heads=0), -1), (dict(n_kv_heads=1025, page_stride=1 << 40), -1), (dict(num_pages=0), -1),
             (dict(num_pages=1 << 27), -1), (dict(page_stride=32 * 2 * 128 - 8), -1), (dict(page_stride=32 * 2 * 128 + 4), -1)]


@pytest.mark.parametrize("kw,code", BAD_PAGES)
def test_pages_are_checked(lib, kw, code):
    k = pages(**kw)
    assert lib.dflash_append_kv(ctypes.byref(k), 4096, 256, 4096, 256, 4096, 1, None) == code
    assert lib.dflash_last_error(None)
    assert lib.dflash_attend_workspace(ctypes.byref(k)) == code
    assert lib.dflash_attend(ctypes.byref(k), *attend_args()) == code
    assert lib.dflash_append_kv(None, 4096, 256, 4096, 256, 4096, 1, None) == -1


def attend_args(**kw):
    a = dict(q=4096, q_stride=8 * 128, page_tables=4096, mpps=4, kv_lens=4096, row_starts=4096, nb=1, n_rows=1, max_new=1, nh=8,
             scale=1.0, window=0, causal=1, out=4096, out_stride=8 * 128, lse=None, workspace=None, workspace_bytes=0, stream=None)
    a.update(kw)
    return list(a.values())


@pytest.mark.parametrize("kw", [
    dict(q=None), dict(out=None), dict(page_tables=None), dict(kv_lens=None), dict(row_starts=None), dict(nb=0), dict(n_rows=-1),
    dict(max_new=-1), dict(mpps=0), dict(mpps=1 << 27), dict(nh=7), dict(nh=0), dict(nh=258), dict(window=-1), dict(scale=0.0),
    dict(scale=-1.0), dict(scale=float("nan")), dict(scale=float("inf")), dict(q_stride=1020), dict(q_stride=1026), dict(dtype=1, q_stride=1028), dict(dtype=1, out_stride=1028),
    dict(out_stride=1000), dict(q=4104), dict(out=4098)])
def test_attend_refuses(lib, kw):
    kw = dict(kw)
    bf16 = kw.pop("dtype", 0) == 1  # (refused before the workspace is asked for, which needs a device)
    k = pages(dtype=1 if bf16 else 0)
    assert lib.dflash_attend(ctypes.byref(k), *attend_args(**kw)) == -1
    assert b"attend" in lib.dflash_last_error(None)


def test_attend_without_rows_is_a_no_op(lib):
    assert lib.dflash_attend(ctypes.byref(pages(dtype=0)), *attend_args(n_rows=0)) == 0


@pytest.mark.parametrize("args,code", [
    ((None, 256, 4096, 256, 4096, 1), -1), ((4096, 256, None, 256, 4096, 1), -1), ((4096, 256, 4096, 256, None, 1), -1),
    ((4096, 256, 4096, 256, 4096, -1), -1), ((4096, 248, 4096, 256, 4096, 1), -1), ((4096, 256, 4096, 260, 4096, 1), -1),
    ((4098, 256, 4096, 256, 4096, 1), -1), ((4096, 256, 4104, 256, 4096, 1), -1), ((None, 0, None, 0, None, 0), 0)])
def test_append_refuses(lib, args, code):
    assert lib.dflash_append_kv(ctypes.byref(pages()), *args, None) == code


def tables_args(**kw):
    a = dict(ctx=4096, new=4096, nb=1, pt=4096, mpps=4, free=4096, n_free=1, begin=4096, end=4096, kv=4096, rs=4096, seq=4096, idx=4096,
             slots=4096, max_rows=1, status=None, stream=None)
    a.update(kw)
    return list(a.values())


@pytest.mark.parametrize("kw,code", [(dict([(n, None)]), -1) for n in ("ctx", "new", "pt", "free", "begin", "end", "kv", "rs", "seq", "idx",
                                                                      "slots")] +
                         [(dict(nb=0), -1), (dict(n_free=-1), -1), (dict(max_rows=-1), -1), (dict(mpps=0), -1), (dict(mpps=1 << 27), -1),
                          (dict(nb=16385), -4), (dict(max_rows=(1 << 30) + 1), -4)])
def test_tables_refuse(lib, kw, code):
    assert lib.dflash_extend_tables(*tables_args(**kw)) == code
    assert b"extend_tables" in lib.dflash_last_error(None)


def sample_args(**kw):
    a = dict(logits=4096, stride=100, dtype=1, rows=1, vocab=100, u=4096, T=None, k=None, p=None, lo=None, tokens=4096, probs=None, stream=None)
    a.update(kw)
    return list(a.values())


@pytest.mark.parametrize("kw,code", [
    (dict(logits=None), -1), (dict(u=None), -1), (dict(tokens=None), -1), (dict(dtype=2), -1), (dict(rows=-1), -1), (dict(vocab=0), -1),
    (dict(stride=99), -1), (dict(logits=4097), -1), (dict(logits=4098, dtype=0), -1), (dict(vocab=752001, stride=752001), -5), (dict(vocab=376001, stride=376001, dtype=0), -5),
    (dict(rows=1 << 28), -4), (dict(rows=0), 0)])
def test_sample_refuses(lib, kw, code):
    assert lib.dflash_sample(*sample_args(**kw)) == code


def test_pages_struct_matches_the_c_compiler(tmp_path):
    import shutil
    import subprocess

    from block_diffusion_drafter_forward_gb300 import _lib
    if shutil.which("gcc") is None:
        pytest.skip("no C compiler")
    fields = [f for f, _ in _lib.dflash_kv_pages._fields_]
    src = tmp_path / "p.c"
    src.write_text('#include <stddef.h>\n#include <stdio.h>\n#include "dflash.h"\nint main(void) { printf("%zu"' +
                   ', sizeof(dflash_kv_pages));\n' + "\n".join(f'printf(" %zu", offsetof(dflash_kv_pages, {f}));' for f in fields) +
                   " return 0; }\n")
    inc = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include")
    subprocess.run(["gcc", "-std=c99", "-I", inc, str(src), "-o", str(tmp_path / "p")], check=True)
    got = [int(v) for v in subprocess.run([str(tmp_path / "p")], capture_output=True, text=True, check=True).stdout.split()]
    assert got == [ctypes.sizeof(_lib.dflash_kv_pages)] + [getattr(_lib.dflash_kv_pages, f).offset for f in fields]


def test_python_calls_refuse_host_tensors_and_wrong_shapes():
    from block_diffusion_drafter_forward_gb300 import PagedKV, extend_tables, sample
    from block_diffusion_drafter_forward_gb300.serve import _addresses, _rows_of
    z = torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError, match="ctx_lens: expected a cuda tensor"):
        extend_tables(z, z, z.view(2, 1), z, z[:1], 4)
    with pytest.raises(ValueError, match="pool: expected a cuda tensor"):
        PagedKV(torch.zeros(2, 1, 2, 1024))
    with pytest.raises(ValueError, match="logits: expected a cuda tensor"):
        sample(torch.zeros(2, 5), torch.zeros(2))
    with pytest.raises(TypeError, match="logits"):
        sample([1.0], torch.zeros(2))
    cpu = torch.device("cpu")
    assert _addresses(cpu, (z, "z", torch.int32, (2,))) == [z.data_ptr()]
    with pytest.raises(TypeError, match="t: expected"):
        _addresses(cpu, ([1, 2], "t", torch.int32, (2,)))
    for t, msg in ((z.float(), "expected torch.int32"), (z[:1], "expected shape"), (torch.zeros(4, dtype=torch.int32)[::2], "contiguous")):
        with pytest.raises(ValueError, match=msg):
            _addresses(cpu, (t, "t", torch.int32, (2,)))
    x = torch.zeros(6, 4, 8)
    assert _rows_of(x[:, 1:3], "x", torch.float32, (6, 2, 8), cpu)[1] == 32
    assert _rows_of(x[:1], "x", torch.float32, (1, 4, 8), cpu)[1] == 32
    for t in (x[:, ::2], x.transpose(0, 1), x[:, :, ::2], x[:1].expand(6, 4, 8)):
        with pytest.raises(ValueError, match="contiguous"):
            _rows_of(t, "x", torch.float32, tuple(t.shape), cpu)


def test_plain_tables_by_hand():
    t, kv, starts, seq, idx, slots, end = R.tables([15, 0], [2, 17], [[4, -1], [-1, -1]], [9, 8, 7, 6], 1, 20)
    assert t.tolist() == [[4, 8], [7, 6]] and kv == [17, 17] and starts == [0, 2, 19] and end == [4]
    assert seq == [0] * 2 + [1] * 17 + [-1] and idx[:4] == [15, 16, 0, 1]
    assert slots[:4] == [4 * 16 + 15, 8 * 16, 7 * 16, 7 * 16 + 1] and slots[18:] == [6 * 16, -1]


def test_plain_sample_by_hand():
    x = np.log(np.array([1.0, 4.0, 2.0, 1.0]))
    assert R.sample(x, 0.0) == (0, pytest.approx(1 / 8))
    assert R.sample(x, 0.126)[0] == 1 and R.sample(x, 0.63)[0] == 2 and R.sample(x, 0.99)[0] == 3
    assert R.sample(x, 0.999, k=3) == (2, pytest.approx(2 / 7))               # equal logits: the lowest index stays
    assert R.sample(x, 0.0, k=3)[0] == 0
    assert R.sample(x, 0.999, p=0.5)[0] == 1 and R.sample(x, 0.999, p=0.51)[0] == 2
    assert R.sample(x, 0.999, lo=0.3)[0] == 2 and R.sample(x, 0.5, T=0.0)[0] == 1
    assert R.sample(np.array([0.0, -np.inf, np.nan]), 0.9) == (0, 1.0)


def test_plain_append_and_rows_are_inverse():
    g = torch.Generator().manual_seed(0)
    k, v = torch.randn(20, 2, 64, generator=g), torch.randn(20, 2, 64, generator=g)
    table = torch.tensor([2, 0], dtype=torch.int32)
    slots = [int(table[i // 16]) * 16 + i % 16 for i in range(20)]
    pool = R.put(torch.zeros(3, 2, 2, 16 * 64), k, v, slots)
    kk, vv = R.rows_of(pool, table, 20)
    assert torch.equal(kk, k.double()) and torch.equal(vv, v.double())
    out, lse, _, _ = R.attend(k[:4].repeat_interleave(2, 1), pool, table[None], [20], [0, 4], True, 1, 1.0)
    assert torch.allclose(out, v[16:].double().repeat_interleave(2, 1))       # a window of one: each row its own value


def test_take_status_refuses_null(lib):
    assert lib.dflash_take_status(None, 4096, None) == -1 and lib.dflash_take_status(4096, None, None) == -1
    assert b"take_status" in lib.dflash_last_error(None)


@pytest.mark.parametrize("kw,code", [(dict(ctx=None), -1), (dict(slots=None), -1), (dict(nb=0), -1), (dict(nb=16385), -4), (dict(mpps=0), -1)])
def test_tables_with_pages_held_refuse(lib, kw, code):
    a = tables_args(**kw)
    assert lib.dflash_extend_tables_ex(*a[:-2], 4096, *a[-2:]) == code
    assert b"extend_tables" in lib.dflash_last_error(None)


def test_sizes_beyond_32_bits_are_refused_or_limited():
    from block_diffusion_drafter_forward_gb300.serve import _i32, _limit
    assert [_limit(n) for n in (5, 0, 2 ** 31 - 1, 2 ** 31, 2 ** 40)] == [5, 0] + [2 ** 31 - 1] * 3
    assert [_limit(n) for n in (-1, -2 ** 31 - 1, -2 ** 32, -2 ** 32 + 7)] == [-1] * 4  # (cut to 32 bits: 0 and 7 among them)
    assert _i32(2 ** 31 - 1, "rows") == 2 ** 31 - 1
    with pytest.raises(ValueError, match="rows: 4294967301 are too many"):
        _i32(2 ** 32 + 5, "rows")
