"""The sparse decode path without a GPU: hand-worked pins of its oracle, the
struct layouts, and the refusals of the C entry points and of the binding."""
import ctypes
import os
import subprocess

import numpy as np
import pytest
import torch

import paged_kv_cache_loc_gb300 as pkv
from oracle import sparse_oracle as S
from paged_kv_cache_loc_gb300 import _lib, build
from test_abi import O, Q, ROOT, fake_cache


@pytest.fixture(scope="module")
def lib():
    build.build()
    return _lib.load()


# ---------------------------------------------------------------------------
# the oracle, by hand
# ---------------------------------------------------------------------------

def test_oracle_tables_by_hand():
    """Pages of 4.  Entry 0 (row 2): 5 cached positions on pages 7, 1, then 4
    new ones: three fill page 1, one opens page 9.  Entry 1 (row 0): one new
    position opens page 3."""
    table = np.array([[-1, -1, -1], [-1, -1, -1], [7, 1, -1]])
    r = S.build_tables([2, 0], [9, 1], [4, 1], table, 4, [8, 9, 3, 5], 1)
    assert r["kv_indptr"].tolist() == [0, 9, 10] and r["qo_indptr"].tolist() == [0, 4, 5]
    assert r["positions"].tolist() == [5, 6, 7, 8, 0]
    assert r["out_cache_loc"].tolist() == [5, 6, 7, 36, 12]
    assert r["req_to_page"].tolist() == [[3, -1, -1], [-1, -1, -1], [7, 1, 9]]
    assert r["free_end"] == 3


def test_oracle_bounds_by_hand():
    """Slot 4 starts page 1 anew, slot 3 widens page 0, a NaN stays."""
    b = np.zeros((2, 1, 2, 2))
    b[0, 0] = [[-1, 5], [2, 6]]
    b[1, 0] = [[-9, -9], [9, 9]]
    got = S.page_bounds(b, np.array([[[0.5, 7]], [[3, -4]], [[np.nan, 1]]]), [3, 4, 5], 4)
    assert got[0, 0].tolist() == [[-1, 5], [2, 7]]
    assert np.isnan(got[1, 0, :, 0]).all() and got[1, 0, :, 1].tolist() == [-4, 1]


def test_oracle_selection_by_hand():
    """Scores 3, 1, 3, 8, 0 for q = (1, -2): page 3 is best, the tie between 0
    and 2 goes to 0; forced pages come first."""
    lo = np.array([[0, -1], [0, 0], [0, -1.5], [0, -4], [0, 0]])
    hi = np.array([[1, 0], [1, 1], [0, 0], [0, 1], [0, 0]])
    b = np.stack([lo, hi], 1)[:, None]
    q = np.array([[[1.0, -2.0]]])
    table = np.arange(5)[None]

    def pick(top_k, first=0, last=0, n=5):
        sel, counts = S.select_pages(b, table, [0], [n], q, 1, top_k, first, last)
        return sel[0, 0, :counts[0, 0]].tolist()
    assert pick(1) == [3] and pick(2) == [0, 3] and pick(3) == [0, 2, 3]
    assert pick(3, 0, 1) == [0, 3, 4] and pick(2, 1, 1) == [0, 4]
    assert pick(7) == [0, 1, 2, 3, 4] and pick(7, n=0) == []
    b[1, 0, 1, 0] = np.nan                               # NaN ranks first
    assert pick(2) == [1, 3]
    two = np.array([[[1.0, -2.0], [-1.0, 0.0]]])         # the group's larger score counts
    b[1, 0] = [[-20, 0], [0, 0]]
    assert S.select_pages(b, table, [0], [5], two, 1, 1, 0, 0)[0][0, 0].tolist() == [1]


def test_oracle_attention_is_softmax_over_the_listed_positions():
    rng = np.random.default_rng(3)
    k, v, q = rng.standard_normal((12, 2, 4)), rng.standard_normal((12, 2, 4)), rng.standard_normal((1, 4, 4))
    table = np.array([[2, 0, 1]])
    sel, counts = np.array([[[0, 2, -1], [1, 2, -1]]]), np.array([[2, 2]])
    o, _ = S.decode_selected(k, v, table, [0], [10], sel, counts, q, 4, 0.5)
    slots = {0: [8, 9, 10, 11, 4, 5], 1: [0, 1, 2, 3, 4, 5]}     # page 2 holds positions 8, 9 of 10
    for h in range(4):
        s = slots[h // 2]
        ref = torch.softmax(torch.tensor(k[s, h // 2] @ q[0, h] * 0.5), 0).numpy() @ v[s, h // 2]
        assert np.allclose(o[0, h], ref, rtol=0, atol=1e-14)


# ---------------------------------------------------------------------------
# layouts and refusals
# ---------------------------------------------------------------------------

def test_struct_layouts_match_the_header(tmp_path):
    fields = {"pkv_tables": _lib.PkvTables, "pkv_pages": _lib.PkvPages}
    prog = '#include <stdio.h>\n#include <stddef.h>\n#include "pkv.h"\nint main(void) {\n'
    want = []
    for name, cls in fields.items():
        prog += f'  printf("%zu ", sizeof({name}));\n'
        want.append(ctypes.sizeof(cls))
        for f, _ in cls._fields_:
            prog += f'  printf("%zu ", offsetof({name}, {f}));\n'
            want.append(getattr(cls, f).offset)
    (tmp_path / "l.c").write_text(prog + "  return 0;\n}\n")
    exe = str(tmp_path / "l")
    subprocess.check_call(["gcc", "-std=c11", "-I", os.path.join(ROOT, "include"), str(tmp_path / "l.c"), "-o", exe])
    assert [int(x) for x in subprocess.check_output([exe]).split()] == want


def tables(**kw):
    t = _lib.PkvTables(0x10000, 0x20000, 8, 16, 0x30000, 0x40000, 0x40004, 100, 64, 0x50000, 0x60000, 0x70000, 0x80000,
                       0x90000)
    for k, v in kw.items():
        setattr(t, k, v)
    return t


@pytest.mark.parametrize("kw", [dict(req_to_page=0), dict(free_start=0), dict(free_end=0), dict(free_end=0x40000),
                                dict(free_pages=0), dict(out_cache_loc=0), dict(max_pages=0), dict(page_size=0),
                                dict(page_size=24), dict(n_free=-1), dict(max_new=-1), dict(max_new=(1 << 30) + 1), dict(max_pages=1 << 30)])
def test_build_tables_refuses(lib, kw):
    assert lib.pkv_build_tables(ctypes.byref(fake_cache()), ctypes.byref(tables(**kw)), None) == _lib.PKV_ERR_ARG


@pytest.mark.parametrize("kw", [dict(batch=-1), dict(batch=65536), dict(num_reqs=0), dict(size=0), dict(max_ctx_len=0),
                                dict(seq_lens=0), dict(req_pool_indices=0)])
def test_build_tables_refuses_the_cache(lib, kw):
    assert lib.pkv_build_tables(ctypes.byref(fake_cache(**kw)), ctypes.byref(tables()), None) == _lib.PKV_ERR_ARG
    assert lib.pkv_build_tables(None, ctypes.byref(tables()), None) == _lib.PKV_ERR_ARG
    assert lib.pkv_build_tables(ctypes.byref(fake_cache()), None, None) == _lib.PKV_ERR_ARG


def pages(**kw):
    p = _lib.PkvPages(0x10000, 0x20000, 16, 16, 8, 1, 1)
    for k, v in kw.items():
        setattr(p, k, v)
    return p


SEL, CNT = ctypes.c_void_p(0xB0000), ctypes.c_void_p(0xC0000)


def calls(lib, c, p, layer=2, q=Q, o=O, heads=32, scale=0.1, sel=SEL, cnt=CNT, n_new=0, k=Q, v=Q, ws=None):
    """Status of select, attend and step for one set of arguments."""
    cc = None if c is None else ctypes.byref(c)
    pp = None if p is None else ctypes.byref(p)
    return [lib.pkv_select_pages(cc, layer, pp, q, heads, sel, cnt, ws, None),
            lib.pkv_paged_decode_selected(cc, layer, pp, sel, cnt, q, o, heads, scale, None),
            lib.pkv_sparse_decode_step(cc, layer, pp, k, v, n_new, q, o, heads, scale, sel, cnt, ws, None)]


BAD = [_lib.PKV_ERR_ARG] * 3


@pytest.mark.parametrize("kw", [dict(req_to_page=0), dict(max_pages=0), dict(max_pages=12), dict(page_size=0),
                                dict(page_size=24), dict(page_size=-16), dict(top_k=0), dict(top_k=1 << 28)])
def test_sparse_calls_refuse_the_pages(lib, kw):
    assert calls(lib, fake_cache(), pages(**kw)) == BAD


@pytest.mark.parametrize("kw", [dict(n_first=-1), dict(n_last=-1), dict(n_first=7, n_last=2)])
def test_selecting_calls_refuse_the_forced_pages(lib, kw):
    """The attention does not read n_first and n_last."""
    select, attend, step = calls(lib, fake_cache(), pages(**kw), scale=float("nan"))
    assert select == step == _lib.PKV_ERR_ARG
    assert calls(lib, fake_cache(batch=0), pages(**kw))[1] == _lib.PKV_OK


@pytest.mark.parametrize("kw", [dict(k_buffer=0), dict(dtype=5), dict(size=0), dict(num_reqs=0), dict(batch=-1),
                                dict(batch=65536), dict(max_len=-1), dict(max_len=257), dict(seq_lens=0),
                                dict(req_pool_indices=0), dict(n_kv_heads=0)])
def test_sparse_calls_refuse_the_cache(lib, kw):
    assert calls(lib, fake_cache(**kw), pages()) == BAD


def test_sparse_calls_refuse_arguments(lib):
    c, p = fake_cache(), pages()
    assert calls(lib, None, p) == BAD and calls(lib, c, None) == BAD
    assert calls(lib, c, p, layer=4) == BAD and calls(lib, c, p, layer=-1) == BAD
    assert calls(lib, c, p, heads=12) == BAD and calls(lib, c, p, heads=0) == BAD
    assert calls(lib, c, p, q=None) == BAD and calls(lib, c, p, q=ctypes.c_void_p(0x900008)) == BAD
    assert calls(lib, c, p, sel=None) == BAD and calls(lib, c, p, cnt=None) == BAD
    assert calls(lib, c, p, o=None)[1:] == BAD[1:] and calls(lib, c, p, o=Q)[1:] == BAD[1:]
    assert calls(lib, c, p, scale=float("inf"))[1:] == BAD[1:]
    assert calls(lib, c, p, n_new=-1)[2] == _lib.PKV_ERR_ARG
    assert calls(lib, c, p, n_new=2, k=None)[2] == _lib.PKV_ERR_ARG
    assert calls(lib, c, pages(page_bounds=0), n_new=2)[2] == _lib.PKV_ERR_ARG
    assert calls(lib, c, p, heads=8 * 16) == [_lib.PKV_ERR_UNSUPPORTED] * 3
    assert calls(lib, fake_cache(head_dim=96), p) == [_lib.PKV_ERR_UNSUPPORTED] * 3
    assert calls(lib, fake_cache(batch=0), p) == [_lib.PKV_OK] * 3       # nothing to do, no CUDA call


def test_attention_refuses_more_kv_heads_than_a_grid_holds(lib):
    """fp32 attention over a group of eight heads takes two CTAs per kv head."""
    def f(n):
        return calls(lib, fake_cache(dtype=_lib.PKV_F32, head_dim=64, n_kv_heads=n, batch=0), pages(), heads=8 * n)
    assert f(32767) == [_lib.PKV_OK] * 3 and f(32768) == [_lib.PKV_OK, _lib.PKV_ERR_ARG, _lib.PKV_ERR_ARG]
    assert calls(lib, fake_cache(n_kv_heads=65536), pages(), heads=65536) == BAD


def test_page_bounds_refuses(lib):
    def f(c=fake_cache(), p=pages(), n=4, layer=2):
        return lib.pkv_page_bounds(ctypes.byref(c), layer, ctypes.byref(p), n, None)
    assert f(n=0) == _lib.PKV_OK
    for bad in (dict(n=-1), dict(layer=4), dict(p=pages(page_bounds=0)), dict(p=pages(page_bounds=0x10008)),
                dict(p=pages(page_size=24)), dict(c=fake_cache(out_cache_loc=0)),
                dict(c=fake_cache(dtype=_lib.PKV_F32, head_dim=2))):
        assert f(**bad) == _lib.PKV_ERR_ARG, bad


def test_select_workspace_bytes(lib):
    f = lib.pkv_select_workspace_bytes
    assert f(0, 8, 100, 16) == f(1, 0, 100, 16) == f(1, 8, 0, 16) == f(1, 8, 100, 0) == 0
    assert f(3, 8, 256, 16) == 3 * 8 * (16 + 1) * 4              # 16 pages: one group
    assert f(3, 8, 257, 16) == 3 * 8 * (32 + 2) * 4
    assert f(65535, 8, 1 << 30, 1) == 65535 * 8 * ((1 << 30) + (1 << 26)) * 4
    assert pkv.select_workspace(3, 8, 257, 16, device="cpu").desc.bytes >= f(3, 8, 257, 16)
    with pytest.raises(ValueError):
        pkv.select_workspace(0, 8, 257, 16, device="cpu")


def test_binding_refuses_cpu_tensors():
    kb = torch.zeros(1, 16, 1, 64)
    cache = pkv.KVCache(k_buffer=kb, v_buffer=kb.clone(), req_to_token=torch.zeros(1, 16, dtype=torch.int32),
                        req_pool_indices=torch.zeros(1, dtype=torch.int32), seq_lens=torch.ones(1, dtype=torch.int32),
                        out_cache_loc=torch.zeros(1, dtype=torch.int32), max_len=1)
    table = torch.zeros(1, 1, dtype=torch.int32)
    pg = pkv.SparsePages.for_cache(cache, table, 16, 4)
    assert pg.page_bounds.shape == (1, 1, 1, 2, 64)
    q = torch.zeros(1, 1, 64)
    sel, cnt = torch.zeros(1, 1, 4, dtype=torch.int32), torch.zeros(1, 1, dtype=torch.int32)
    word = torch.zeros(1, dtype=torch.int32)
    for f in (lambda: pkv.select_pages(cache, 0, pg, q), lambda: pkv.page_bounds(cache, 0, pg),
              lambda: pkv.paged_decode_selected(cache, 0, pg, q, sel, cnt),
              lambda: pkv.sparse_decode_step(cache, 0, pg, q, q, q),
              lambda: pkv.build_tables(cache, table, 16, word, word, word.clone())):
        with pytest.raises(ValueError, match="CUDA"):
            f()
