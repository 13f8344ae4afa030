"""The life of a cache's pages and chunk attention without a GPU: hand-worked
pins of their oracle, the struct layout, and the refusals of the C entry points
and of the binding."""
import ctypes
import os
import subprocess

import numpy as np
import pytest
import torch

import paged_kv_cache_loc_gb300 as pkv
from oracle import pages_oracle as P
from paged_kv_cache_loc_gb300 import _lib, build
from test_abi import O, Q, ROOT, fake_cache


@pytest.fixture(scope="module")
def lib():
    build.build()
    return _lib.load()


# ---------------------------------------------------------------------------
# the oracle, by hand
# ---------------------------------------------------------------------------

def pool(n_slots, layers=2):
    k = np.arange(layers * n_slots).reshape(layers, n_slots, 1)
    return k, k + 1000


def test_oracle_copy_by_hand():
    """Pages of 2: page 3 takes page 0's rows; -1 and a page itself are passed over."""
    k, v = pool(8)
    bounds = np.arange(8).reshape(2, 4)
    got = P.copy_pages(k, v, bounds, 2, [0, -1, 2], [3, 1, 2])
    assert got[0][:, :, 0].tolist() == [[0, 1, 2, 3, 4, 5, 0, 1], [8, 9, 10, 11, 12, 13, 8, 9]]
    assert got[1][0, 6:, 0].tolist() == [1000, 1001] and got[2].tolist() == [[0, 1, 2, 0], [4, 5, 6, 4]]


def test_oracle_fork_by_hand():
    """Pages of 2.  Row 1 takes 3 positions of row 0 (pages 2, 0): page 2 is
    shared, page 0's first slot goes to page 3; row 2 takes 2: page 2 alone."""
    k, v = pool(8, 1)
    table = np.array([[2, 0], [-1, -1], [-1, -1]])
    tokens = np.full((3, 4), -1)
    k, v, b, table, tokens, shares, end = P.fork(k, v, None, 2, table, tokens, np.zeros(4, int), [1, 2], [0, 0], [3, 2], [9, 3, 1], 1)
    assert table.tolist() == [[2, 0], [2, 3], [2, -1]] and shares.tolist() == [0, 0, 2, 0] and end == 2
    assert k[0, :, 0].tolist() == [0, 1, 2, 3, 4, 5, 0, 7]
    assert tokens.tolist() == [[-1] * 4, [4, 5, 6, -1], [4, 5, -1, -1]]


def test_oracle_release_by_hand():
    """Rows 0 (pages 5, 1, 4) and 1 (5, 2) give up what lies behind 1 and 0
    positions of pages of 2: 5 is left to row 0, 1, 2 and 4 are free."""
    table, shares, free, end = P.release(np.array([[5, 1, 4], [5, 2, -1]]), np.array([0, 0, 0, 0, 0, 1]), 2, [0, 1], [6, 4], [1, 0],
                                         np.array([9, 9, 9, 9, 0, 3]), 4)
    assert table.tolist() == [[5, -1, -1], [-1, -1, -1]] and shares.tolist() == [0] * 6
    assert free.tolist() == [9, 1, 2, 4, 0, 3] and end == 1


def test_oracle_compact_by_hand():
    """Pages 0, 2 and 5 of 6 are used: 5 goes to 1."""
    k, v = pool(6, 1)
    table, tokens = np.array([[5, 2, 0, -1]]), np.array([[5, 2, 0, -1, 7]])
    k, v, b, table, tokens, shares, free, remap = P.compact(k, v, None, 1, table, tokens, np.array([0, 0, 3, 0, 0, 7]),
                                                            np.array([4, 3, 1, 4]), 1)
    assert remap.tolist() == [0, 1, 2, 3, 4, 1] and table.tolist() == [[1, 2, 0, -1]] and tokens.tolist() == [[1, 2, 0, -1, 7]]
    assert shares.tolist() == [0, 7, 3, 0, 0, 0] and free.tolist() == [4, 3, 4, 5] and k[0, :, 0].tolist() == [0, 5, 2, 3, 4, 5]


def test_oracle_chunk_by_hand():
    """Two rows at the end of three positions, weights 1/2, 1/2 and 1/3 each;
    not causal 1/3 each; more rows than positions: the first sees nothing."""
    k, v = np.zeros((4, 1, 1)), np.array([1.0, 2.0, 6.0, 9.0]).reshape(4, 1, 1)
    table = np.array([[1, 0]])                        # positions 0, 1, 2 at slots 2, 3, 0
    q = np.ones((3, 1, 1))
    o, _, _ = P.chunk(k, v, table, 2, [0], [3], [0, 2], q, True, 1.0, np.full((3, 1, 1), 7.0))
    assert np.allclose(o[:, 0, 0], [7.5, 16 / 3, 7.0])
    o, _, _ = P.chunk(k, v, table, 2, [0], [3], [0, 2], q, False, 1.0, np.zeros((3, 1, 1)))
    assert np.allclose(o[:, 0, 0], [16 / 3, 16 / 3, 0])
    o, _, _ = P.chunk(k, v, table, 2, [0], [2], [0, 3], q, True, 1.0, np.ones((3, 1, 1)))
    assert np.allclose(o[:, 0, 0], [0, 6, 7.5])


# ---------------------------------------------------------------------------
# the C ABI
# ---------------------------------------------------------------------------

def test_struct_layout_matches_header(tmp_path):
    prog = tmp_path / "layout.c"
    prog.write_text(r'''
#include <stdio.h>
#include <stddef.h>
#include "pkv.h"
int main(void) {
  printf("%zu %zu %zu %zu %zu %zu\n", sizeof(pkv_page_state), offsetof(pkv_page_state, shares), offsetof(pkv_page_state, free_end),
         offsetof(pkv_page_state, n_free), offsetof(pkv_page_state, req_to_token), offsetof(pkv_page_state, page_bounds));
  return 0;
}''')
    exe = tmp_path / "layout"
    subprocess.check_call(["gcc", "-std=c11", "-I", os.path.join(ROOT, "include"), str(prog), "-o", str(exe)])
    got = [int(x) for x in subprocess.check_output([str(exe)]).split()]
    T = _lib.PkvPageState
    assert got == [ctypes.sizeof(T), T.shares.offset, T.free_end.offset, T.n_free.offset, T.req_to_token.offset, T.page_bounds.offset]


def state(**kw):
    s = _lib.PkvPageState(req_to_page=0x1000, max_pages=8, page_size=16, shares=0x2000, free_pages=0x3000, free_start=0x4000,
                          free_end=0x4004, n_free=4, req_to_token=0x5000, page_bounds=0)
    for k, v in kw.items():
        setattr(s, k, v)
    return s


PTR = ctypes.c_void_p(0x1000)


def test_copy_refuses(lib):
    def call(c=None, ps=16, bounds=None, src=PTR, dst=PTR, n=1):
        return lib.pkv_copy_pages(ctypes.byref(c or fake_cache()), ps, bounds, src, dst, n, None)

    assert lib.pkv_copy_pages(None, 16, None, PTR, PTR, 1, None) == _lib.PKV_ERR_ARG
    assert call(n=0) == _lib.PKV_OK                       # nothing to do: no CUDA call
    for kw in (dict(n=-1), dict(ps=0), dict(ps=-16), dict(src=None), dict(dst=None), dict(bounds=ctypes.c_void_p(0x1008)),
               dict(c=fake_cache(size=17)), dict(c=fake_cache(size=0)), dict(c=fake_cache(k_buffer=0)), dict(c=fake_cache(dtype=9)),
               dict(c=fake_cache(n_layers=0)), dict(c=fake_cache(v_buffer=0x1004))):
        assert call(**kw) == _lib.PKV_ERR_ARG, kw
    # pages whose chunks pass 31 bits
    assert call(c=fake_cache(size=1 << 24, n_layers=64), ps=1 << 24) == _lib.PKV_ERR_ARG


@pytest.mark.parametrize("name", ["fork", "release", "compact"])
def test_state_refusals(lib, name):
    def call(c=None, t=None, null=False):
        c, t = ctypes.byref(c or fake_cache()), ctypes.byref(t or state())
        if null:
            t = None
        if name == "fork":
            return lib.pkv_fork_requests(c, t, PTR, None)
        if name == "release":
            return lib.pkv_release_pages(c, t, None, None)
        ws = _lib.PkvWorkspace()
        return lib.pkv_compact_pages(c, t, PTR, PTR, ctypes.byref(ws), None)

    assert call(null=True) == _lib.PKV_ERR_ARG
    for kw in (dict(max_pages=0), dict(page_size=0), dict(page_size=7), dict(n_free=-1), dict(req_to_page=0), dict(shares=0),
               dict(free_start=0), dict(free_pages=0), dict(max_pages=1 << 28)):
        assert call(t=state(**kw)) == _lib.PKV_ERR_ARG, kw
    for kw in (dict(num_reqs=0), dict(size=0), dict(max_ctx_len=0)):
        assert call(c=fake_cache(**kw)) == _lib.PKV_ERR_ARG, kw
    assert call() == _lib.PKV_ERR_ARG                     # addresses that no GPU reaches


def test_workspace_sizes(lib):
    assert lib.pkv_compact_workspace_bytes(0) == 0 and lib.pkv_compact_workspace_bytes(-1) == 0
    assert lib.pkv_compact_workspace_bytes(1 << 32) == 0
    for n in (1, 2, 7, 1000):
        assert lib.pkv_compact_workspace_bytes(n) >= 4 * (1 + n // 2 * 2)


def test_chunk_refuses(lib):
    def call(c=None, layer=0, table=PTR, max_pages=512, ps=16, q=Q, o=O, n_q=4, heads=32, max_q=4, scale=0.1, ws=None):
        return lib.pkv_paged_chunk(ctypes.byref(c or fake_cache(qo_indptr=0x9000)), layer, table, max_pages, ps, q, o, n_q, heads, max_q, 1,
                                   scale, ws, None)

    assert lib.pkv_paged_chunk(None, 0, PTR, 8, 16, Q, O, 4, 32, 4, 1, 0.1, None, None) == _lib.PKV_ERR_ARG
    for kw in (dict(layer=-1), dict(layer=99), dict(table=None), dict(max_pages=0), dict(ps=0), dict(ps=13), dict(q=None), dict(o=None),
               dict(o=Q), dict(n_q=-1), dict(heads=0), dict(heads=31), dict(max_q=-1), dict(max_q=65535 * 64), dict(scale=float("nan")),
               dict(scale=float("inf")), dict(max_pages=1), dict(q=ctypes.c_void_p(0x1004)),
               dict(c=fake_cache(qo_indptr=0)), dict(c=fake_cache(qo_indptr=0x9000, seq_lens=0)), dict(c=fake_cache(qo_indptr=0x9000, batch=-1)),
               dict(c=fake_cache(qo_indptr=0x9000, batch=70000))):
        assert call(**kw) == _lib.PKV_ERR_ARG, kw
    assert call(heads=24) == _lib.PKV_ERR_UNSUPPORTED                 # groups of 3
    assert call(c=fake_cache(qo_indptr=0x9000, head_dim=96)) == _lib.PKV_ERR_UNSUPPORTED
    for c in (fake_cache(qo_indptr=0x9000, batch=0),):
        assert call(c=c) == _lib.PKV_OK
    assert call(n_q=0) == _lib.PKV_OK and call(max_q=0) == _lib.PKV_OK
    assert call() in (_lib.PKV_ERR_ARG, _lib.PKV_ERR_CUDA)           # addresses that no GPU reaches, or no GPU


def test_binding_refuses_cpu_tensors():
    k = torch.zeros(1, 32, 1, 64, dtype=torch.bfloat16)
    i = torch.zeros(2, dtype=torch.int32)
    c = pkv.KVCache(k_buffer=k, v_buffer=k, req_to_token=i[None], req_pool_indices=i, seq_lens=i, qo_indptr=i)
    for call in (lambda: pkv.copy_pages(c, 16, i, i), lambda: pkv.fork_requests(c, i[None], 16, i, i, i, i[:1], i[1:]),
                 lambda: pkv.release_pages(c, i[None], 16, i, i, i[:1], i[1:]), lambda: pkv.compact_pages(c, i[None], 16, i, i, i[:1]),
                 lambda: pkv.paged_chunk(c, 0, i[None], 16, torch.zeros(2, 1, 64, dtype=torch.bfloat16), 1)):
        with pytest.raises(ValueError, match="CUDA"):
            call()
