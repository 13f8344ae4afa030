"""The sparse decode path on the GPU against its fp64 oracle.

Whole numbers (tables, selections, counts) and copies (bounds) are equal.  The
attention's tolerance per output o of a softmax-weighted mean of values v, with
A the largest sum_c |q_c k_c| * scale of a pair: a score is a sum of D products
in fp32, each partial sum off by 2^-23 of its size at most, so weights are off
by the factor exp(2 D 2^-23 A) at most, and the sums over n positions by n
2^-23 more; 2^-15 covers weights that a bf16 product takes as two bf16 parts;
the output rounding is half a step, 2^-8 |o| in bf16 and 2^-24 |o| in fp32:
  |err| <= max|v| (4 D 2^-23 A + 4 n 2^-23 + [bf16] 2^-15) + half a step.
"""
import dataclasses
import math

import numpy as np
import pytest
import torch

import paged_kv_cache_loc_gb300 as pkv
from oracle import sparse_oracle as S
from paged_kv_cache_loc_gb300 import _lib, build
from paged_kv_cache_loc_gb300 import pool as pkv_pool

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f32": torch.float32}


@pytest.fixture(scope="module", autouse=True)
def gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    build.build()
    torch.cuda.set_device(0)
    pkv.last_device_error()
    yield
    torch.cuda.synchronize()


def dev(a, dtype=torch.int32):
    return torch.from_numpy(np.ascontiguousarray(a)).to(dtype).cuda()


def host(t):
    return t.double().cpu().numpy() if t.is_floating_point() else t.cpu().numpy().astype(np.int64)


def clean():
    status, detail = pkv.last_device_error()
    assert status == _lib.PKV_OK, detail


def error():
    status, detail = pkv.last_device_error()
    assert status == _lib.PKV_ERR_INDEX
    return detail


def ws_for(batch, kv, max_len, ps, device="cuda"):
    return pkv.select_workspace(max(1, batch), kv, max(1, max_len), ps, device=device)


# ---------------------------------------------------------------------------
# build_tables
# ---------------------------------------------------------------------------

@dataclasses.dataclass
class Tables:
    cache: object
    table: object
    free: object
    start: object
    end: object
    positions: object
    q: object
    ps: int

    def run(self, q_lens=True, **kw):
        pkv.build_tables(self.cache, self.table, self.ps, self.free, self.start, self.end, self.positions,
                         self.q if q_lens else None, **kw)


def tables_case(rng, lens, q_lens, ps, spare=7, extra_free=3, skip=4):
    lens, q_lens = np.asarray(lens), np.asarray(q_lens)
    batch = len(lens)
    rows = rng.permutation(batch + 2)[:batch]
    old = lens - q_lens
    need = -(-lens // ps) - -(-old // ps)
    n_pages = int((-(-lens // ps)).sum()) + extra_free + 1
    perm = rng.permutation(n_pages)
    max_pages = int((-(-lens // ps)).max(initial=0)) + 2
    table = np.full((batch + 2, max_pages), -7)
    at = 0
    for b in range(batch):
        m = -(-int(old[b]) // ps)
        table[rows[b], :m] = perm[at:at + m]
        at += m
    free = np.r_[np.full(skip, -5), perm[at:at + int(need.sum()) + extra_free]]
    n_new = int(q_lens.sum())
    kb = torch.empty(1, n_pages * ps, 1, 8, device="cuda", dtype=torch.bfloat16)
    cache = pkv.KVCache(k_buffer=kb, v_buffer=kb, req_to_token=torch.full((batch + 2, max_pages * ps), -3, dtype=torch.int32, device="cuda"),
                        req_pool_indices=dev(rows), seq_lens=dev(lens), out_cache_loc=torch.full((n_new + spare,), -9, dtype=torch.int32, device="cuda"),
                        kv_indptr=torch.zeros(batch + 1, dtype=torch.int32, device="cuda"), qo_indptr=torch.zeros(batch + 1, dtype=torch.int32, device="cuda"))
    t = Tables(cache, dev(table), dev(free), dev([skip]), dev([-1]), torch.full((n_new + spare,), -9, dtype=torch.int32, device="cuda"), dev(q_lens), ps)
    want = S.build_tables(rows, lens, q_lens, table, ps, free, skip)
    want["req_to_token"] = np.full((batch + 2, max_pages * ps), -3)
    at = 0
    for b in range(batch):
        for p in range(old[b], lens[b]):
            want["req_to_token"][rows[b], p] = want["out_cache_loc"][at]
            at += 1
    return t, want, n_new


def check_tables(t, want, n_new, token_table=True):
    assert np.array_equal(host(t.table), want["req_to_page"])
    assert int(t.end) == want["free_end"]
    assert np.array_equal(host(t.cache.kv_indptr), want["kv_indptr"])
    assert np.array_equal(host(t.cache.qo_indptr), want["qo_indptr"])
    for got, name in ((t.cache.out_cache_loc, "out_cache_loc"), (t.positions, "positions")):
        assert np.array_equal(host(got)[:n_new], want[name]), name
        assert (host(got)[n_new:] == -9).all(), "entries behind the last token were written"
    assert np.array_equal(host(t.cache.req_to_token), want["req_to_token"] if token_table else np.full_like(want["req_to_token"], -3))


@pytest.mark.parametrize("ps", [1, 3, 16, 64])
@pytest.mark.parametrize("batch,hi_old,hi_new", [(1, 40, 1), (1, 0, 700), (7, 90, 30), (64, 300, 1), (600, 20, 9), (5000, 9, 3)])
def test_build_tables(ps, batch, hi_old, hi_new):
    rng = np.random.default_rng(ps * 1000 + batch + hi_new)
    q = rng.integers(0 if batch > 1 else hi_new, hi_new + 1, batch)
    t, want, n = tables_case(rng, rng.integers(0, hi_old + 1, batch) + q, q, ps)
    t.run()
    clean()
    check_tables(t, want, n)


def test_build_tables_one_long_prompt_among_empty_entries():
    """More tokens than one CTA owns, entries without tokens on both sides."""
    rng = np.random.default_rng(5)
    q = np.zeros(40, np.int64)
    q[17], q[30] = 9000, 5
    t, want, n = tables_case(rng, q + rng.integers(0, 50, 40), q, 16, spare=0)
    t.run(token_table=False)
    clean()
    check_tables(t, want, n, token_table=False)


def test_build_tables_decode_lengths_are_optional():
    """Without q_lens each entry that is not empty has one new token."""
    rng = np.random.default_rng(6)
    lens = rng.integers(0, 70, 33)
    t, want, n = tables_case(rng, lens, (lens > 0).astype(np.int64), 16)
    t.run(q_lens=False)
    clean()
    check_tables(t, want, n)


def test_build_tables_at_the_largest_batch():
    rng = np.random.default_rng(7)
    q = rng.integers(0, 3, 65535)
    t, want, n = tables_case(rng, q + rng.integers(0, 4, 65535), q, 2)
    t.run()
    clean()
    check_tables(t, want, n)


def test_build_tables_replayed_from_a_graph_over_a_growing_context():
    """Steps replayed from a graph, the free list's place carried from step to
    step and the lengths growing in place, equal the oracle's steps."""
    rng = np.random.default_rng(8)
    lens = rng.integers(1, 30, 9)
    t, _, _ = tables_case(rng, lens, np.ones(9, np.int64), 4, spare=0, extra_free=60)
    table, start, free, rows = host(t.table), int(t.start), host(t.free), host(t.cache.req_pool_indices)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        t.run(q_lens=False, stream=side)
        t.start.copy_(t.end)
        t.cache.seq_lens.add_(1)
    for step in range(6):
        want = S.build_tables(rows, lens, np.ones(9, np.int64), table, 4, free, start)
        g.replay()
        torch.cuda.synchronize()
        assert np.array_equal(host(t.table), want["req_to_page"]) and int(t.start) == want["free_end"]
        assert np.array_equal(host(t.cache.out_cache_loc), want["out_cache_loc"])
        table, start, lens = want["req_to_page"], want["free_end"], lens + 1
    clean()


def test_build_tables_reports_bad_entries_and_serves_the_others():
    for what, detail in (("row", 99), ("len", 1 << 20), ("q", 77), ("negative", -4)):
        rng = np.random.default_rng(9)
        lens, q = np.array([20, 33, 7, 50]), np.array([4, 9, 7, 1])
        q_ok = q.copy()
        q_ok[1] = 0
        lens_ok = lens.copy()
        lens_ok[1] = 0
        t, want, n = tables_case(rng, lens_ok, q_ok, 8)
        rows, lens, q = host(t.cache.req_pool_indices), lens, q
        if what == "row":
            rows[1] = detail
        elif what == "len":
            lens[1] = detail
        elif what == "q":
            q[1] = detail
        else:
            lens[1] = detail
        t.cache.req_pool_indices, t.cache.seq_lens, t.q = dev(rows), dev(lens), dev(q)
        t.run()
        assert error() == detail
        check_tables(t, want, n)


def test_build_tables_free_list_runs_out():
    """The tokens without a page get slot -1, nothing else changes."""
    rng = np.random.default_rng(10)
    t, want, n = tables_case(rng, np.array([10, 21]), np.array([10, 21]), 8, extra_free=0)
    t.free = t.free[:-2].contiguous()                    # 5 pages needed, 3 left: entry 1 gets one
    t.run()
    assert error() == -300001
    loc, full = host(t.cache.out_cache_loc)[:n], want["out_cache_loc"]
    assert np.array_equal(loc[:18], full[:18]) and (loc[18:] == -1).all()
    assert int(t.end) == t.free.numel()
    row = host(t.table)[host(t.cache.req_pool_indices)[1]]
    assert row[0] == want["req_to_page"][host(t.cache.req_pool_indices)[1], 0] and (row[1:3] == -1).all()


def test_build_tables_too_many_tokens_and_bad_pages():
    rng = np.random.default_rng(11)
    t, want, n = tables_case(rng, np.array([10, 21]), np.array([10, 21]), 8, spare=0)
    t.cache.out_cache_loc, t.positions = t.cache.out_cache_loc[:12].contiguous(), t.positions[:12].contiguous()
    t.run()
    assert error() == 31
    assert np.array_equal(host(t.cache.out_cache_loc), want["out_cache_loc"][:12])
    for where in ("free", "table"):
        t, want, n = tables_case(rng, np.array([10, 21]), np.array([10, 19]), 8)
        if where == "free":
            t.free[4] = 12345
        else:
            t.table[t.cache.req_pool_indices[1].long(), 0] = 12345
        t.run()
        assert error() == 12345
        bad = np.zeros(n, bool)
        bad[:8] = where == "free"                        # the first page taken: entry 0's positions 0 .. 7
        bad[10:16] = where == "table"                    # entry 1's positions 2 .. 7
        assert np.array_equal(host(t.cache.out_cache_loc)[:n], np.where(bad, -1, want["out_cache_loc"]))
    t, want, n = tables_case(rng, np.array([10]), np.array([10]), 8)
    t.start.fill_(-2)
    t.run()
    assert error() == -2 and (host(t.cache.out_cache_loc)[:n] == -1).all()


@pytest.mark.parametrize("batch,ps,room", [(2, 8, 12), (2, 8, 0), (7, 16, 1), (300, 4, 900), (5000, 2, 3000), (40, 1, 39)])
def test_build_tables_pages_of_tokens_without_a_slot(batch, ps, room):
    """With more tokens than out_cache_loc holds, the page table, the prefix sums
    and the free list's place are those of all tokens: no page is lost, and no
    column keeps a page of another request.  A list that runs out gives -1."""
    rng = np.random.default_rng(batch + room)
    q = rng.integers(0, 40, batch)
    q[-1] = max(q[-1], room - int(q[:-1].sum()) + 1)
    t, want, n = tables_case(rng, q + rng.integers(0, 30, batch), q, ps, spare=0, extra_free=0)
    assert n > room
    for cut in (0, 3):                                   # pages that the list lacks
        free = t.free[:t.free.numel() - cut].contiguous()
        table, loc, positions = t.table.clone(), t.cache.out_cache_loc[:room].clone(), t.positions[:room].clone()
        cache = dataclasses.replace(t.cache, out_cache_loc=loc if room else None)
        pkv.build_tables(cache, table, ps, free, t.start, t.end, positions if room else None, t.q)
        detail = error()
        assert detail == n or (cut and -300000 - batch < detail <= -300000)
        gone = host(t.free)[free.numel():]
        full = np.where(np.isin(want["req_to_page"], gone) & (host(t.table) != want["req_to_page"]), -1, want["req_to_page"])
        assert np.array_equal(host(table), full)
        assert int(t.end) == want["free_end"] - cut
        assert np.array_equal(host(cache.kv_indptr), want["kv_indptr"]) and np.array_equal(host(cache.qo_indptr), want["qo_indptr"])
        slots = want["out_cache_loc"][:room]
        assert np.array_equal(host(loc), np.where(np.isin(slots // ps, gone), -1, slots))
        assert np.array_equal(host(positions), want["positions"][:room])


# ---------------------------------------------------------------------------
# page_bounds
# ---------------------------------------------------------------------------

def pool(rng, n_layers, n_pages, ps, kv, d, dtype):
    def make():
        x = torch.from_numpy(rng.standard_normal((n_layers, n_pages * ps, kv, d), dtype=np.float32))
        return x.to(DT[dtype]).cuda()
    return make(), make()


@pytest.mark.parametrize("dtype,kv,d,ps", [("bf16", 8, 128, 16), ("bf16", 2, 64, 16), ("bf16", 1, 128, 1), ("bf16", 3, 64, 7),
                                           ("bf16", 16, 128, 100), ("f32", 8, 128, 16), ("f32", 1, 64, 5), ("bf16", 1, 8, 40)])
def test_page_bounds(dtype, kv, d, ps):
    """Runs that start and end anywhere in a page, in any page order, more
    tokens than a CTA takes, runs longer than a warp; the other layer's bounds
    and untouched pages stay."""
    rng = np.random.default_rng(ps)
    n_pages = 300
    k, v = pool(rng, 2, n_pages, ps, kv, d, dtype)
    loc = []
    for page in rng.permutation(n_pages)[:250]:
        a = 0 if rng.random() < 0.5 else int(rng.integers(0, ps))
        loc += [page * ps + i for i in range(a, int(rng.integers(a, ps)) + 1)]
    cache = pkv.KVCache(k_buffer=k, v_buffer=v, req_to_token=dev(np.zeros((1, 1))), req_pool_indices=dev([0]), out_cache_loc=dev(loc))
    pg = pkv.SparsePages.for_cache(cache, dev(np.zeros((1, 1))), ps, 4)
    pg.page_bounds.copy_(torch.from_numpy(rng.standard_normal(pg.page_bounds.shape)))
    before = host(pg.page_bounds)
    pkv.page_bounds(cache, 1, pg)
    clean()
    assert np.array_equal(host(pg.page_bounds)[0], before[0])
    assert np.array_equal(host(pg.page_bounds)[1], S.page_bounds(before[1], host(k)[1][loc], loc, ps))


def test_page_bounds_bad_slots_and_nan():
    """A slot outside the pool is reported and skipped; a NaN key stays in its
    channel's bounds, infinities too."""
    rng = np.random.default_rng(1)
    k, v = pool(rng, 1, 8, 4, 2, 64, "bf16")
    k[0, 9, 0, 3], k[0, 9, 1, 5], k[0, 9, 1, 6] = math.nan, math.inf, -math.inf
    loc = [8, 9, 10, -1, 11, 32, 20, 21]
    cache = pkv.KVCache(k_buffer=k, v_buffer=v, req_to_token=dev(np.zeros((1, 1))), req_pool_indices=dev([0]), out_cache_loc=dev(loc[:3] + loc[6:]))
    pg = pkv.SparsePages.for_cache(cache, dev(np.zeros((1, 1))), 4, 4)
    want = S.page_bounds(host(pg.page_bounds)[0], host(k)[0][loc[:3] + loc[6:]], loc[:3] + loc[6:], 4)
    pkv.page_bounds(cache, 0, pg)
    clean()
    assert np.array_equal(host(pg.page_bounds)[0], want, equal_nan=True)
    cache.out_cache_loc = dev(loc)
    pkv.page_bounds(cache, 0, pg)
    assert error() in (-1, 32)
    want = S.page_bounds(want, host(k)[0][loc[:3] + [11, 20, 21]], loc[:3] + [11, 20, 21], 4)
    assert np.array_equal(host(pg.page_bounds)[0], want, equal_nan=True)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("ps,n_pages,stay", [(4, 30, 0.6), (16, 80, 0.5), (16, 900, 0.8), (70, 60, 0.9)])
def test_page_bounds_of_slots_with_gaps(dtype, ps, n_pages, stay):
    """A page's new tokens in ascending slots that are not consecutive, a page
    begun anew or not, spread over several CTAs, with the write and without; a
    slot that stands twice in a row (not the page's first) counts as one page's."""
    rng = np.random.default_rng(ps + n_pages)
    k, v = pool(rng, 1, n_pages, ps, 2, 64, dtype)
    loc = []
    for page in rng.permutation(n_pages):
        slots = page * ps + np.flatnonzero(rng.random(ps) < stay)
        loc += list(slots) + [x for x in slots[-1:] if x % ps and rng.random() < 0.2]
    cache = pkv.KVCache(k_buffer=k, v_buffer=v, req_to_token=dev(np.zeros((1, 1))), req_pool_indices=dev([]), seq_lens=dev([]), out_cache_loc=dev(loc))
    pg = pkv.SparsePages.for_cache(cache, dev(np.zeros((1, 1))), ps, 4)
    pg.page_bounds.copy_(torch.from_numpy(rng.standard_normal(pg.page_bounds.shape)))
    before = pg.page_bounds.clone()
    pkv.page_bounds(cache, 0, pg)
    clean()
    assert np.array_equal(host(pg.page_bounds)[0], S.page_bounds(host(before)[0], host(k)[0][loc], loc, ps))
    pg.page_bounds.copy_(before)
    kn, vn = (torch.randn(len(loc), 2, 64, device="cuda").to(DT[dtype]) for _ in range(2))
    pkv.sparse_decode_step(cache, 0, pg, kn, vn, torch.zeros(0, 8, 64, dtype=DT[dtype], device="cuda"))
    clean()
    assert np.array_equal(host(pg.page_bounds)[0], S.page_bounds(host(before)[0], host(kn), loc, ps))


def test_page_bounds_and_selection_behind_4_gb():
    """Bounds rows whose offset passes 2^32 bytes, in the second layer."""
    rng = np.random.default_rng(2)
    n_pages = (1 << 19) + 64
    k = torch.zeros(2, n_pages, 8, 128, dtype=torch.bfloat16, device="cuda")
    loc = np.r_[n_pages - 40:n_pages]
    k[1, loc] = torch.randn(40, 8, 128, device="cuda").bfloat16()
    cache = pkv.KVCache(k_buffer=k, v_buffer=k, req_to_token=dev(np.zeros((1, 1))), req_pool_indices=dev([0]), seq_lens=dev([40]),
                        out_cache_loc=dev(loc), max_len=40)
    pg = pkv.SparsePages.for_cache(cache, dev(loc[None]), 1, 6)
    assert pg.page_bounds.numel() * 2 > 1 << 32
    pkv.page_bounds(cache, 1, pg)
    q = torch.randn(1, 32, 128, device="cuda").bfloat16()
    sel, counts = pkv.select_pages(cache, 1, pg, q, workspace=ws_for(1, 8, 40, 1))
    clean()
    assert torch.equal(pg.page_bounds[1, -40:, :, 0], k[1, -40:]) and not pg.page_bounds[0].any()
    want, _ = S.select_pages(host(pg.page_bounds[1, -40:]), np.arange(40)[None], [0], [40], host(q), 1, 6, 1, 1)
    assert np.array_equal(host(sel), want)
    o = pkv.paged_decode_selected(cache, 1, pg, q, sel, counts)
    clean()
    kk = host(k[1, -40:])
    ref, reach = S.decode_selected(kk, kk, np.arange(40)[None], [0], [40], want, host(counts), host(q), 1, 128 ** -0.5)
    close(o, ref, reach, kk, 6, "bf16")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_step_on_rows_behind_4_gb(dtype):
    """The pool's rows, and with them every row that the step writes and reads,
    lie past 2^32 bytes."""
    rng = np.random.default_rng(50)
    size = (1 << 21 if dtype == "bf16" else 1 << 20) + 2048
    ps, kv, d, n = 16, 8, 128, 1000
    k, v = (torch.zeros(1, size, kv, d, dtype=DT[dtype], device="cuda") for _ in range(2))
    assert (size - 2048) * kv * d * k.element_size() >= 1 << 32
    table = (size - 2048) // ps + rng.permutation(128)[None, :63]
    p = np.arange(n)
    slots = table[0, p // ps] * ps + p % ps
    k[0, dev(slots).long()], v[0, dev(slots).long()] = (torch.randn(n, kv, d, device="cuda").to(DT[dtype]) for _ in range(2))
    cache = pkv.KVCache(k_buffer=k, v_buffer=v, req_to_token=dev(np.zeros((1, 1))), req_pool_indices=dev([0]), seq_lens=dev([n]),
                        out_cache_loc=dev(slots[:-1]), max_len=n)
    pg = pkv.SparsePages.for_cache(cache, dev(table), ps, 12)
    pkv.page_bounds(cache, 0, pg)
    cache.out_cache_loc = dev(slots[-1:])
    kn, vn, q = (torch.randn(1, h, d, device="cuda").to(DT[dtype]) for h in (kv, kv, 32))
    o, sel, counts = pkv.sparse_decode_step(cache, 0, pg, kn, vn, q, workspace=ws_for(1, kv, n, ps))
    clean()
    lo = size - 2048
    assert torch.equal(k[0, dev(slots[-1:]).long()], kn) and not k[0, :lo].any() and not v[0, :lo].any()
    kk, vv = host(k[0, lo:]), host(v[0, lo:])
    bounds = S.page_bounds(np.zeros((128, kv, 2, d)), kk[slots - lo], slots - lo, ps)
    assert np.array_equal(host(pg.page_bounds[0, lo // ps:]), bounds) and not pg.page_bounds[0, :lo // ps].any()
    want = S.select_pages(bounds, table - lo // ps, [0], [n], host(q), ps, 12, 1, 1)
    assert np.array_equal(host(sel), want[0])
    ref, reach = S.decode_selected(kk, vv, table - lo // ps, [0], [n], *want, host(q), ps, d ** -0.5)
    close(o, ref, reach, vv, 12 * ps, dtype)


# ---------------------------------------------------------------------------
# select_pages
# ---------------------------------------------------------------------------

def bounds_of(rng, n_pages, kv, d, dtype, spread=1.0):
    mid, half = rng.standard_normal((n_pages, kv, 1, d)), np.abs(rng.standard_normal((n_pages, kv, 1, d))) * spread
    b = torch.from_numpy(np.concatenate([mid - half, mid + half], 2).astype(np.float32)).to(DT[dtype])
    return b[None].contiguous().cuda()


def select_case(rng, dtype, heads, kv, d, ps, lens, top_k, first=1, last=1, bounds=None, q=None, shared_row=False):
    batch, max_len = len(lens), max(1, int(np.max(lens)))
    np_max = -(-max_len // ps)
    n_pages = (1 if shared_row else batch) * np_max + 3
    rows = np.full(batch, 1) if shared_row else rng.permutation(batch + 1)[:batch]
    table = np.full((batch + 1, np_max + 1), 0)
    perm = rng.permutation(n_pages)
    for i, r in enumerate(np.unique(rows)):
        table[r, :np_max] = perm[i * np_max:(i + 1) * np_max]
    if bounds is None:
        bounds = bounds_of(rng, n_pages, kv, d, dtype)
    elif callable(bounds):
        bounds = bounds(n_pages)
    k = torch.zeros(1, n_pages * ps, kv, d, dtype=DT[dtype], device="cuda")
    cache = pkv.KVCache(k_buffer=k, v_buffer=k, req_to_token=dev(np.zeros((1, 1))), req_pool_indices=dev(rows), seq_lens=dev(lens), max_len=max_len)
    pg = pkv.SparsePages(bounds, dev(table), ps, top_k, first, last)
    if q is None:
        q = torch.from_numpy(rng.standard_normal((batch, heads, d)).astype(np.float32)).to(DT[dtype]).cuda()
    return cache, pg, q, (table, rows, lens)


def check_select(cache, pg, q, where, **kw):
    kv = cache.k_buffer.shape[2]
    ws = ws_for(len(where[2]), kv, cache.max_len, pg.page_size)
    ws.buffer.fill_(0xAB)
    sel, counts = pkv.select_pages(cache, 0, pg, q, workspace=ws, **kw)
    clean()
    want = S.select_pages(host(pg.page_bounds)[0], *where, host(q), pg.page_size, pg.top_k, pg.n_first, pg.n_last)
    assert np.array_equal(host(counts), want[1])
    assert np.array_equal(host(sel), want[0])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("group,kv,d,ps", [(1, 8, 128, 16), (2, 3, 64, 1), (4, 2, 128, 24), (8, 1, 64, 16), (8, 2, 128, 5), (4, 8, 64, 16),
                                           (1, 1, 64, 2), (2, 4, 128, 128)])
def test_select_pages(dtype, group, kv, d, ps):
    rng = np.random.default_rng(group * 100 + ps)
    lens = np.array([0, 1, ps, ps + 1, 8 * ps, 8 * ps + 1, 31 * ps - 1, 77 * ps, 260 * ps + 1])
    for top_k, first, last in ((8, 1, 1), (1, 0, 0), (5, 0, 2), (20, 3, 0), (4, 2, 2)):
        check_select(*select_case(rng, dtype, group * kv, kv, d, ps, lens, top_k, first, last))


def test_select_pages_long_contexts():
    rng = np.random.default_rng(21)
    check_select(*select_case(rng, "bf16", 8, 2, 128, 4, np.array([40000, 33333, 3]), 200, 1, 2))
    check_select(*select_case(rng, "bf16", 8, 2, 64, 1, np.array([70000]), 64, 0, 0))
    check_select(*select_case(rng, "f32", 4, 2, 64, 1, np.array([20000, 9]), 1000, 0, 0))


def test_select_pages_without_a_workspace_when_every_page_fits():
    rng = np.random.default_rng(22)
    cache, pg, q, where = select_case(rng, "bf16", 8, 2, 64, 16, np.array([128, 0, 1]), 8)
    sel, counts = pkv.select_pages(cache, 0, pg, q)
    clean()
    assert host(counts).tolist() == [[8, 8], [0, 0], [1, 1]]
    assert host(sel)[0, 0].tolist() == list(range(8)) and (host(sel)[1] == -1).all()
    cache.max_len = 129
    with pytest.raises(pkv.PkvError) as e:
        pkv.select_pages(cache, 0, pg, q)
    assert e.value.status == _lib.PKV_ERR_WORKSPACE
    with pytest.raises(pkv.PkvError) as e:
        pkv.select_pages(cache, 0, pg, q, workspace=pkv.Workspace(1, 1, 1, 1))
    assert e.value.status == _lib.PKV_ERR_WORKSPACE


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("kinds", [1, 2, 7])
@pytest.mark.parametrize("pages", [60, 2000])
def test_select_pages_ties_go_to_the_lowest(dtype, kinds, pages):
    """Pages with the same bounds, from few undecided ones to thousands."""
    rng = np.random.default_rng(kinds)
    kind = bounds_of(rng, kinds, 2, 64, dtype)[0]

    def bounds(n):
        return kind[torch.from_numpy(rng.integers(0, kinds, n)).cuda()][None].contiguous()
    check_select(*select_case(rng, dtype, 4, 2, 64, 1, np.array([pages, pages - 9]), 33, 1, 1, bounds=bounds))


def test_select_pages_zero_queries_and_zero_bounds():
    rng = np.random.default_rng(24)
    zero = torch.zeros(2, 8, 64, dtype=torch.bfloat16, device="cuda")
    check_select(*select_case(rng, "bf16", 8, 2, 64, 2, np.array([300, 2000]), 9, 0, 1, q=zero))
    check_select(*select_case(rng, "bf16", 8, 2, 64, 2, np.array([300, 2000]), 9, 0, 1, bounds=lambda n: torch.zeros(1, n, 2, 2, 64, dtype=torch.bfloat16, device="cuda")))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("pages", [40, 900])
def test_select_pages_zero_times_infinity_ranks_first(dtype, pages):
    """Queries of zeros over bounds of which some are infinite: those scores
    are NaN, the others zero."""
    rng = np.random.default_rng(pages)
    q = torch.zeros(2, 8, 64, dtype=DT[dtype], device="cuda")
    q[1, 3, 5] = 1.0

    def bounds(n):
        b = bounds_of(rng, n, 2, 64, dtype)
        b[0, torch.from_numpy(rng.permutation(n)[:5]).cuda(), 1, 1, 7] = math.inf
        return b
    check_select(*select_case(rng, dtype, 8, 2, 64, 1, np.array([pages, pages - 3]), 9, 0, 1, bounds=bounds, q=q))


def test_page_bounds_of_rotated_keys():
    """The bounds are those of what the cache holds: here after the fused
    rotary write."""
    rng = np.random.default_rng(48)
    k, v = pool(rng, 1, 10, 8, 2, 64, "bf16")
    loc = np.r_[16:24, 40:43, 9:11]
    cache = pkv.KVCache(k_buffer=k, v_buffer=v, req_to_token=dev(np.zeros((1, 1))), req_pool_indices=dev([0]), out_cache_loc=dev(loc))
    pg = pkv.SparsePages.for_cache(cache, dev(np.zeros((1, 1))), 8, 4)
    angle = torch.arange(32, device="cuda")[None] * torch.arange(20, device="cuda")[:, None] * 0.01
    pkv.rope_kv_write(cache, 0, torch.randn(13, 2, 64, device="cuda").bfloat16(), torch.randn(13, 2, 64, device="cuda").bfloat16(),
                      torch.stack([angle.cos(), angle.sin()], -1).contiguous(), dev(np.arange(13)))
    pkv.page_bounds(cache, 0, pg)
    clean()
    assert np.array_equal(host(pg.page_bounds)[0], S.page_bounds(np.zeros((10, 2, 2, 64)), host(k)[0][loc], loc, 8))


def test_build_tables_a_row_named_twice_leaves_the_others_exact():
    """What such a row's tables hold is unspecified; the pages taken, the sums,
    the positions and the other rows are not."""
    rng = np.random.default_rng(52)
    q = np.array([9, 14, 9, 3])
    t, want, n = tables_case(rng, q + np.array([0, 5, 0, 20]), q, 4)
    rows = host(t.cache.req_pool_indices)
    rows[2] = rows[0]
    t.cache.req_pool_indices = dev(rows)
    t.run()
    clean()
    assert np.array_equal(host(t.cache.kv_indptr), want["kv_indptr"]) and int(t.end) == want["free_end"]
    assert np.array_equal(host(t.positions)[:n], want["positions"])
    single = np.r_[9:23, 32:35]                          # the tokens of entries 1 and 3
    assert np.array_equal(host(t.cache.out_cache_loc)[single], want["out_cache_loc"][single])
    assert np.array_equal(host(t.table)[rows[[1, 3]]], want["req_to_page"][rows[[1, 3]]])


def test_page_bounds_a_slot_given_twice_leaves_the_other_pages_exact():
    rng = np.random.default_rng(53)
    k, v = pool(rng, 1, 12, 4, 2, 64, "bf16")
    loc = np.r_[8:12, 9, 20:24, 20:22, 40:43]
    cache = pkv.KVCache(k_buffer=k, v_buffer=v, req_to_token=dev(np.zeros((1, 1))), req_pool_indices=dev([0]), out_cache_loc=dev(loc))
    pg = pkv.SparsePages.for_cache(cache, dev(np.zeros((1, 1))), 4, 4)
    pkv.page_bounds(cache, 0, pg)
    clean()
    want = S.page_bounds(np.zeros((12, 2, 2, 64)), host(k)[0][40:43], np.r_[40:43], 4)
    others = [p for p in range(12) if p not in (2, 5)]
    assert np.array_equal(host(pg.page_bounds)[0][others], want[others])


def test_build_tables_of_an_empty_batch():
    rng = np.random.default_rng(49)
    t, _, _ = tables_case(rng, np.array([5]), np.array([5]), 4)
    none = torch.zeros(0, dtype=torch.int32, device="cuda")
    t.cache.req_pool_indices = t.cache.seq_lens = t.q = none
    t.cache.kv_indptr, t.cache.qo_indptr = (torch.full((1,), 7, dtype=torch.int32, device="cuda") for _ in range(2))
    t.run()
    clean()
    assert int(t.end) == int(t.start) and int(t.cache.kv_indptr) == 0 and int(t.cache.qo_indptr) == 0
    assert (host(t.cache.out_cache_loc) == -9).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_select_pages_scores_that_32_bits_do_not_tell_apart(dtype):
    """Large channels that cancel, and differences of one small channel far
    below the rounding of the sum: the order is the 64-bit one."""
    rng = np.random.default_rng(25)
    q = torch.ones(1, 2, 128, device="cuda")
    q[:, :, 64:] = -1

    def bounds(n):
        b = torch.full((1, n, 1, 2, 128), 4096.0, device="cuda")      # +4096 * 64 - 4096 * 64
        b[:, :, :, :, 5] += torch.from_numpy(rng.permutation(n)).cuda()[None, :, None, None] * 32.0
        b[:, :, :, :, 9] = torch.from_numpy(rng.integers(0, 2, n)).cuda()[None, :, None, None] * 2.0 ** -12
        return b.to(DT[dtype])
    check_select(*select_case(rng, dtype, 2, 1, 128, 1, np.array([900]), 100, 0, 0, bounds=bounds, q=q.to(DT[dtype])))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_select_pages_scores_are_within_their_error_bound(dtype):
    """What the order of the selection rests on: a 32-bit score is off from the
    exact one by 2^-16 of max_h sum |q| times the largest |bound| at most (the
    scores' order-preserving keys stand at the start of the workspace in the form
    with two launches, which the size of the batch chooses)."""
    batch, kv, group, d, n = 256, 8, 4, 128, 320
    gen = torch.Generator("cuda").manual_seed(56)

    def rnd(*shape):
        return torch.randn(*shape, generator=gen, device="cuda")
    ramp = 2.0 ** torch.linspace(-10, 10, d, device="cuda")
    for kind in ("alike", "cancelling", "of all sizes", "two large", "ramps"):
        q, b = rnd(batch, kv * group, d), rnd(n, kv, 2, d)
        if kind == "cancelling":
            q, b = q.sign() * (1 + 0.01 * q), b * 0.01 + 1000
        elif kind == "of all sizes":
            q, b = q * torch.exp(3 * rnd(batch, kv * group, d)), b * torch.exp(4 * rnd(n, kv, 1, d))
        elif kind == "two large":
            b[..., 7], b[..., 9] = 3e4, -3e4
            q[..., 9] = q[..., 7]
        elif kind == "ramps":
            q, b = q.sign() * ramp.flip(0), b.sign() * ramp
        q, b = q.to(DT[dtype]), b.to(DT[dtype])
        b = torch.stack([b.amin(2), b.amax(2)], 2)[None].contiguous()
        k = torch.zeros(1, n, kv, d, dtype=DT[dtype], device="cuda")
        cache = pkv.KVCache(k_buffer=k, v_buffer=k, req_to_token=dev(np.zeros((1, 1))), req_pool_indices=dev(np.zeros(batch)),
                            seq_lens=dev(np.full(batch, n)), max_len=n)
        pg = pkv.SparsePages(b, dev(np.arange(n)[None]), 1, 8)
        ws = ws_for(batch, kv, n, 1)
        pkv.select_pages(cache, 0, pg, q, workspace=ws)
        clean()
        at = (ws.desc.base - ws.buffer.data_ptr())
        keys = ws.buffer[at:at + batch * kv * n * 4].view(torch.int32).view(batch, kv, n)
        score = torch.where(keys < 0, keys & 0x7fffffff, ~keys).view(torch.float32).double()
        x, y = q.double().view(batch, kv, group * d).transpose(0, 1).reshape(kv, batch * group, d), b[0].double().permute(1, 2, 3, 0)
        exact = (x.clamp(max=0) @ y[:, 0] + x.clamp(min=0) @ y[:, 1]).view(kv, batch, group, n).amax(2).transpose(0, 1)
        bound = 2.0 ** -16 * q.double().abs().sum(-1).view(batch, kv, group).amax(2) * b.double().abs().max()
        assert ((score - exact).abs() <= bound[:, :, None]).all(), kind


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_select_pages_nan_infinite_and_huge_bounds(dtype):
    rng = np.random.default_rng(26)
    for fill in (math.nan, math.inf, 3e38, -math.inf):
        for few in (3, 700):
            def bounds(n):
                b = bounds_of(rng, n, 2, 64, dtype)
                at = torch.from_numpy(rng.permutation(n)[:few]).cuda()
                if fill == -math.inf:
                    b[0, at, :, 0, 3] = fill
                else:
                    b[0, at, :, 1, 3] = fill
                    if fill != fill:
                        b[0, at, :, 0, 3] = fill
                return b
            check_select(*select_case(rng, dtype, 4, 2, 64, 1, np.array([1500, 40]), 17, 1, 1, bounds=bounds))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("pages", [40, 250, 900])
@pytest.mark.parametrize("where", ["any", "first", "unasked"])
def test_select_pages_beside_a_few_outlying_bounds(dtype, pages, where):
    """A few pages with one finite channel of 1e10 to 1e30 (any pages, the page
    that is always in, a channel where q is 0): the error bound leaves all the
    others undecided, and their order is that of their own scores."""
    rng = np.random.default_rng(54)
    for size in (1e10, 1e17, 1e20, 1e30):
        cache, pg, q, (table, rows, lens) = select_case(rng, dtype, 4, 2, 64, 1, np.array([pages, 30]), 17, 1, 1)
        if where == "unasked":
            q[:, :, 3] = 0
        for i, page in enumerate([0] if where == "first" else [5, 17, 30]):
            phys = int(table[rows[0], page])
            pg.page_bounds[0, phys, :, 1, 3] = size * (i + 1)
            pg.page_bounds[0, phys, :, 0, 4] = -size * (i + 2)
        check_select(cache, pg, q, (table, rows, lens))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("pages", [700, 3000, 9000])
@pytest.mark.parametrize("steps,other", [(1, None), (200, None), (200, math.nan), (200, -math.inf), (3, math.inf), (200, 1e30)])
def test_select_pages_many_alike(dtype, pages, steps, other):
    """More pages than a list holds whose scores are 2^20 and `steps` different
    remainders of 2^-6 (the upper half of an fp64 score is the same), a few pages
    with one other bound among them: the 64-bit order, ties to the lowest.  Small
    contexts in one launch, long ones with their scores in the workspace."""
    rng = np.random.default_rng(pages + steps)
    q = torch.zeros(2, 4, 64, device="cuda")
    q[:, :, 0] = 1.0
    q[:, ::2, 1], q[:, 1::2, 1] = 1.0, -1.0

    def bounds(n):
        b = torch.zeros(1, n, 2, 2, 64, device="cuda")
        b[..., 0] = 2.0 ** 20
        b[..., 1] = dev(rng.integers(0, steps, (n, 2, 1)), torch.float32) * 2.0 ** -6
        if other is not None:
            b[0, dev(rng.permutation(n)[:7]).long(), :, 1, 1] = other
        return b.to(DT[dtype])
    check_select(*select_case(rng, dtype, 4, 2, 64, 1, np.array([pages, pages - 5]), 100, 1, 1, bounds=bounds, q=q.to(DT[dtype])))


def test_select_pages_queries_of_one_request():
    """The queries of a prompt: entries that name one row with growing lengths."""
    rng = np.random.default_rng(27)
    check_select(*select_case(rng, "bf16", 8, 2, 128, 4, 500 + np.arange(37), 12, 1, 1, shared_row=True))


@pytest.mark.parametrize("dtype,group,kv,d", [("bf16", 1, 8, 64), ("bf16", 2, 8, 128), ("bf16", 4, 8, 128), ("bf16", 8, 8, 128), ("f32", 8, 8, 128), ("f32", 1, 8, 64)])
def test_select_pages_of_many_entries(dtype, group, kv, d):
    """Large batches, whose scores have a launch of their own: runs of entries
    of one request of any length (queries of prompts whose last pages differ),
    short and empty contexts among them."""
    rng = np.random.default_rng(group * d)
    batch, ps = 700, 4
    cache, pg, q, (table, rows, lens) = select_case(rng, dtype, group * kv, kv, d, ps, rng.integers(0, 60 * ps, batch), 7, 1, 1)
    at = 0
    while at < batch:
        n = int(rng.integers(1, 40))
        row = int(rng.integers(0, batch))
        rows[at:at + n] = row
        lens[at:at + n] = np.minimum(60 * ps - 1, int(rng.integers(0, 50 * ps)) + np.arange(n))[:len(lens[at:at + n])]
        at += n + int(rng.integers(0, 5))
    perm = rng.permutation(pg.page_bounds.shape[1])[:table.shape[1]]
    table[:, :] = perm[None]                             # every row holds pages: its own order of the same ones
    for r in range(table.shape[0]):
        table[r] = np.roll(perm, r)
    cache.req_pool_indices, cache.seq_lens, cache.max_len = dev(rows), dev(lens), 60 * ps
    pg = dataclasses.replace(pg, req_to_page=dev(table))
    check_select(cache, pg, q, (table, rows, lens))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_select_pages_of_a_batch_of_long_contexts(dtype):
    """Two launches with more pages than a small batch's, ties among them."""
    rng = np.random.default_rng(29)
    lens = np.array([5000, 4100, 10, 4999, 3000, 0, 4500, 2500])
    kind = bounds_of(rng, 40, 8, 64, dtype)[0]
    check_select(*select_case(rng, dtype, 16, 8, 64, 1, lens, 100, 1, 1))
    check_select(*select_case(rng, dtype, 16, 8, 64, 1, lens, 100, 1, 1, bounds=lambda n: kind[torch.from_numpy(rng.integers(0, 40, n)).cuda()][None].contiguous()))


def test_select_pages_reports_bad_device_data():
    rng = np.random.default_rng(28)
    cache, pg, q, (table, rows, lens) = select_case(rng, "bf16", 8, 2, 64, 4, np.array([200, 180, 90]), 6)
    ws = ws_for(3, 2, 200, 4)
    want = S.select_pages(host(pg.page_bounds)[0], table, rows, lens, host(q), 4, 6, 1, 1)[0]
    for field, value in (("req_pool_indices", 44), ("seq_lens", -3), ("seq_lens", 201)):
        t = getattr(cache, field).clone()
        t[1] = value
        sel, counts = pkv.select_pages(dataclasses.replace(cache, **{field: t}), 0, pg, q, workspace=ws)
        assert error() == value
        assert np.array_equal(host(sel)[[0, 2]], want[[0, 2]])
        if value != 201:
            assert (host(counts)[1] == 0).all() and (host(sel)[1] == -1).all()
    t = pg.req_to_page.clone()
    t[int(rows[1]), 7] = 1 << 20
    sel, _ = pkv.select_pages(cache, 0, dataclasses.replace(pg, req_to_page=t), q, workspace=ws)
    assert error() == 1 << 20
    assert np.array_equal(host(sel)[[0, 2]], want[[0, 2]])


# ---------------------------------------------------------------------------
# paged_decode_selected
# ---------------------------------------------------------------------------

def close(o, ref, reach, v, n, dtype):
    bf16 = dtype == "bf16"
    d = ref.shape[-1]
    tol = np.abs(v).max() * (4 * d * 2.0 ** -23 * reach + 4 * n * 2.0 ** -23 + (2.0 ** -15 if bf16 else 0.0))
    err = np.abs(host(o) - ref) - (2.0 ** -8 if bf16 else 2.0 ** -24) * np.abs(ref)
    assert np.isfinite(host(o)).all() and err.max() <= tol, (err.max(), tol)


def attend_case(rng, dtype, heads, kv, d, ps, lens, top_k, poison=True):
    """A pool whose slots outside the contexts hold NaN, and lists of pages in
    ascending order with the last page among them."""
    batch, max_len = len(lens), max(1, int(np.max(lens)))
    pages = -(-np.asarray(lens) // ps)
    n_pages = int(pages.sum()) + 4
    k, v = pool(rng, 2, n_pages, ps, kv, d, dtype)
    rows, perm = rng.permutation(batch + 2)[:batch], rng.permutation(n_pages)
    table = np.zeros((batch + 2, -(-max_len // ps) + 1), np.int64)
    used, at = np.zeros(n_pages * ps, bool), 0
    for b in range(batch):
        table[rows[b], :pages[b]] = perm[at:at + pages[b]]
        at += int(pages[b])
        p = np.arange(lens[b])
        used[table[rows[b], p // ps] * ps + p % ps] = True
    if poison:
        k[:, dev(~used, torch.bool)] = math.nan
        v[:, dev(~used, torch.bool)] = math.nan
    sel, counts = np.full((batch, kv, top_k), -1), np.zeros((batch, kv), np.int64)
    for b in range(batch):
        for g in range(kv):
            c = min(top_k, int(pages[b]))
            pick = rng.permutation(pages[b])[:c]
            if c and pages[b] - 1 not in pick:
                pick[0] = pages[b] - 1
            sel[b, g, :c], counts[b, g] = np.sort(pick), c
    cache = pkv.KVCache(k_buffer=k, v_buffer=v, req_to_token=dev(np.zeros((1, 1))), req_pool_indices=dev(rows), seq_lens=dev(lens), max_len=max_len)
    q = torch.from_numpy(rng.standard_normal((batch, heads, d)).astype(np.float32)).to(DT[dtype]).cuda()
    return cache, pkv.SparsePages(None, dev(table), ps, top_k), q, table, rows, sel, counts


def check_attend(case, lens, dtype, layer=1, **kw):
    cache, pg, q, table, rows, sel, counts = case
    o = pkv.paged_decode_selected(cache, layer, pg, q, dev(sel), dev(counts), **kw)
    clean()
    k, v = np.nan_to_num(host(cache.k_buffer[layer])), np.nan_to_num(host(cache.v_buffer[layer]))
    scale = kw.get("sm_scale") or q.shape[2] ** -0.5
    ref, reach = S.decode_selected(k, v, table, rows, lens, sel, counts, host(q), pg.page_size, scale)
    close(o, ref, reach, v, int(counts.max()) * pg.page_size, dtype)
    return o


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("group,kv,d,ps,top_k", [(4, 8, 128, 16, 8), (1, 8, 128, 16, 5), (2, 3, 64, 7, 9), (8, 1, 128, 1, 40), (8, 2, 64, 24, 6),
                                                 (4, 2, 64, 16, 64), (2, 8, 128, 128, 3), (1, 1, 64, 33, 2), (8, 8, 128, 16, 20)])
def test_attend(dtype, group, kv, d, ps, top_k):
    """Lengths from none to long ones; the slots behind each context are NaN."""
    rng = np.random.default_rng(ps + group)
    lens = np.array([0, 1, ps, ps + 1, 3 * ps - 1, 11 * ps + 2, 40 * ps + 1])
    case = attend_case(rng, dtype, group * kv, kv, d, ps, lens, top_k)
    o = check_attend(case, lens, dtype)
    assert (o[0] == 0).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("batch,top_k,ps", [(1, 900, 1), (1, 256, 16), (1, 1, 16), (200, 3, 16), (3, 2, 700)])
def test_attend_splits_and_long_lists(dtype, batch, top_k, ps):
    """One entry over a whole cluster, lists longer than a stage, many entries
    without a split, pages longer than a stage."""
    rng = np.random.default_rng(top_k)
    lens = rng.integers(1, 2 * ps * top_k, batch)
    lens[0] = ps * top_k + ps // 2
    check_attend(attend_case(rng, dtype, 8, 2, 128, ps, lens, top_k), lens, dtype, sm_scale=0.2)


def test_attend_lists_in_any_order_and_twice():
    """An unsorted list gives the same sums; a page listed twice counts twice."""
    rng = np.random.default_rng(31)
    lens = np.array([100, 37])
    case = list(attend_case(rng, "bf16", 4, 1, 64, 8, lens, 6))
    case[5] = np.array([[[12, 0, 5, 5, 3, -1]], [[4, 2, 0, 3, -1, -1]]])
    case[6] = np.array([[5], [4]])
    check_attend(case, lens, "bf16")


def test_attend_equals_the_dense_decode_when_every_page_is_listed():
    rng = np.random.default_rng(32)
    lens = np.array([300, 128, 77])
    cache, pg, q, table, rows, sel, counts = attend_case(rng, "bf16", 32, 8, 128, 16, lens, 19)
    o = check_attend((cache, pg, q, table, rows, sel, counts), lens, "bf16")
    dense = pkv.paged_decode_pages(cache, 1, pg.req_to_page, 16, q, workspace=pkv.Workspace(3, 32, 128, 64))
    clean()
    assert (o.float() - dense.float()).abs().max() <= 2 ** -6


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_attend_scores_of_any_size(dtype):
    """Scores far from zero (the running maximum moves), and a scale of 0."""
    rng = np.random.default_rng(33)
    lens = np.array([500, 40])
    case = attend_case(rng, dtype, 8, 2, 64, 8, lens, 30)
    check_attend(case, lens, dtype, sm_scale=3.0)
    cache, pg, q, table, rows, sel, counts = case
    o = pkv.paged_decode_selected(cache, 1, pg, q, dev(sel), dev(counts), sm_scale=0.0)
    v = np.nan_to_num(host(cache.v_buffer[1]))
    ref, _ = S.decode_selected(np.zeros_like(v), v, table, rows, lens, sel, counts, host(q), 8, 1.0)
    close(o, ref, 0.0, v, 240, dtype)


def test_attend_nan_and_infinite_values_reach_their_own_head_only():
    """A NaN value in a selected position is not lost, and the other kv head is
    not touched by it."""
    rng = np.random.default_rng(34)
    lens = np.array([64])
    cache, pg, q, table, rows, sel, counts = attend_case(rng, "bf16", 8, 2, 64, 8, lens, 8)
    slot = int(table[rows[0], 3]) * 8 + 2
    cache.v_buffer[1, slot, 0, 7] = math.nan
    o = pkv.paged_decode_selected(cache, 1, pg, q, dev(sel), dev(counts))
    clean()
    assert torch.isnan(o[0, :4, 7]).all() and torch.isfinite(o[0, 4:]).all()
    assert torch.isfinite(o[0, :4, :7]).all() and torch.isfinite(o[0, :4, 8:]).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("what", [math.inf, -math.inf])
def test_attend_an_infinite_value_makes_its_channel_not_finite(dtype, what):
    """An infinite value in a selected position (bf16 weights go in as two parts,
    so it may come out as NaN): not finite in its channel of its group's outputs,
    every other output has the bits that it has without it."""
    rng = np.random.default_rng(55)
    lens = np.array([64, 300])
    cache, pg, q, table, rows, sel, counts = attend_case(rng, dtype, 8, 2, 64, 8, lens, 8)
    want = pkv.paged_decode_selected(cache, 1, pg, q, dev(sel), dev(counts)).clone()
    for b, page in ((0, 3), (1, int(sel[1, 0, 4]))):
        cache.v_buffer[1, int(table[rows[b], page]) * 8 + 2, 0, 7] = what
    o = pkv.paged_decode_selected(cache, 1, pg, q, dev(sel), dev(counts))
    clean()
    assert not torch.isfinite(o[:, :4, 7]).any()
    o[:, :4, 7] = want[:, :4, 7]
    assert torch.equal(o, want)


def test_attend_reports_bad_device_data():
    rng = np.random.default_rng(35)
    lens = np.array([60, 50, 40])
    cache, pg, q, table, rows, sel, counts = attend_case(rng, "bf16", 8, 2, 64, 4, lens, 6)
    good = pkv.paged_decode_selected(cache, 1, pg, q, dev(sel), dev(counts))
    clean()

    def run(cache=cache, pg=pg, sel=sel, counts=counts):
        o = pkv.paged_decode_selected(cache, 1, pg, q, dev(sel), dev(counts))
        detail = error()
        assert torch.equal(o[[0, 2]], good[[0, 2]])
        return o, detail
    for field, value in (("req_pool_indices", -1), ("seq_lens", 1000), ("seq_lens", -5)):
        t = getattr(cache, field).clone()
        t[1] = value
        assert run(cache=dataclasses.replace(cache, **{field: t}))[1] == value
    bad = counts.copy()
    bad[1, 0] = 7
    assert run(counts=bad)[1] == 7
    bad = sel.copy()
    bad[1, 1, 2] = 13                                    # the context has pages 0 .. 12
    o, detail = run(sel=bad)
    assert detail == 13
    less = np.delete(sel[1, 1], 2)
    sel2, counts2 = sel.copy(), counts.copy()
    sel2[1, 1, :5], counts2[1, 1] = less, 5
    assert (o[1].float() - pkv.paged_decode_selected(cache, 1, pg, q, dev(sel2), dev(counts2))[1].float()).abs().max() <= 2 ** -7
    t = pg.req_to_page.clone()
    t[int(rows[1]), int(sel[1, 0, 0])] = 1 << 24
    assert run(pg=dataclasses.replace(pg, req_to_page=t))[1] == 1 << 24


# ---------------------------------------------------------------------------
# the step, and the calls together
# ---------------------------------------------------------------------------

def step_case(rng, dtype, heads, kv, d, ps, lens, top_k, n_layers=2):
    cache, pg, q, table, rows, _, _ = attend_case(rng, dtype, heads, kv, d, ps, lens, top_k, poison=False)
    batch = len(lens)
    pos = lens - 1
    loc = table[rows, pos // ps] * ps + pos % ps
    cache.out_cache_loc = dev(loc)
    pg = pkv.SparsePages.for_cache(cache, pg.req_to_page, ps, top_k, 1, 2)
    for layer in range(2):                               # the bounds of what is cached
        b = np.zeros(pg.page_bounds.shape[1:])
        for i in range(batch):
            p = np.arange(lens[i] - 1)
            slots = table[rows[i], p // ps] * ps + p % ps
            b = S.page_bounds(b, host(cache.k_buffer[layer, dev(slots).long()]), slots, ps)
        pg.page_bounds[layer].copy_(torch.from_numpy(b))
    kn, vn = (torch.from_numpy(rng.standard_normal((batch, kv, d)).astype(np.float32)).to(DT[dtype]).cuda() for _ in range(2))
    return cache, pg, q, kn, vn, table, rows, loc


def check_step(case, lens, dtype, run):
    cache, pg, q, kn, vn, table, rows, loc = case
    k, v, b = host(cache.k_buffer), host(cache.v_buffer), host(pg.page_bounds)
    k[1, loc], v[1, loc] = host(kn), host(vn)
    b[1] = S.page_bounds(b[1], host(kn), loc, pg.page_size)
    o, sel, counts = run()
    clean()
    assert np.array_equal(host(cache.k_buffer), k) and np.array_equal(host(cache.v_buffer), v)
    assert np.array_equal(host(pg.page_bounds), b)
    want = S.select_pages(b[1], table, rows, lens, host(q), pg.page_size, pg.top_k, pg.n_first, pg.n_last)
    assert np.array_equal(host(sel), want[0]) and np.array_equal(host(counts), want[1])
    ref, reach = S.decode_selected(k[1], v[1], table, rows, lens, *want, host(q), pg.page_size, q.shape[2] ** -0.5)
    close(o, ref, reach, v[1], pg.top_k * pg.page_size, dtype)
    return o, sel, counts


@pytest.mark.parametrize("dtype,group,kv,d,ps", [("bf16", 4, 8, 128, 16), ("bf16", 8, 2, 64, 8), ("bf16", 1, 3, 128, 5), ("f32", 4, 2, 64, 16), ("f32", 2, 8, 128, 1)])
def test_sparse_decode_step(dtype, group, kv, d, ps):
    """The step against the oracle and bit for bit against the four calls."""
    rng = np.random.default_rng(ps)
    lens = np.array([1, ps + 1, 9 * ps, 33 * ps + 1, 200 * ps - 3 if ps > 3 else 190])
    case = step_case(rng, dtype, group * kv, kv, d, ps, lens, 12)
    cache, pg, q, kn, vn = case[:5]
    ws = ws_for(len(lens), kv, cache.max_len, ps)
    copy = dataclasses.replace(cache, k_buffer=cache.k_buffer.clone(), v_buffer=cache.v_buffer.clone())
    pg2 = dataclasses.replace(pg, page_bounds=pg.page_bounds.clone())
    o, sel, counts = check_step(case, lens, dtype, lambda: pkv.sparse_decode_step(cache, 1, pg, kn, vn, q, workspace=ws))
    pkv.kv_write(copy, 1, kn, vn)
    pkv.page_bounds(copy, 1, pg2)
    sel2, counts2 = pkv.select_pages(copy, 1, pg2, q, workspace=ws)
    o2 = pkv.paged_decode_selected(copy, 1, pg2, q, sel2, counts2)
    clean()
    assert torch.equal(sel, sel2) and torch.equal(counts, counts2) and torch.equal(o, o2) and torch.equal(pg.page_bounds, pg2.page_bounds)


def test_step_of_a_prompt_chunk():
    """64 new tokens of one request, each an entry that sees the positions up
    to its own (some pages are begun, others opened)."""
    rng = np.random.default_rng(41)
    ps, n, old = 8, 64, 501
    table = rng.permutation(90)[None, :80]
    k, v = pool(rng, 2, 90, ps, 2, 128, "bf16")
    lens = old + 1 + np.arange(n)
    loc = table[0, (lens - 1) // ps] * ps + (lens - 1) % ps
    cache = pkv.KVCache(k_buffer=k, v_buffer=v, req_to_token=dev(np.zeros((1, 1))), req_pool_indices=dev(np.zeros(n)), seq_lens=dev(lens),
                        out_cache_loc=dev(loc), max_len=int(lens.max()))
    pg = pkv.SparsePages.for_cache(cache, dev(table), ps, 10, 1, 2)
    p = np.arange(old)
    slots = table[0, p // ps] * ps + p % ps
    pg.page_bounds[1].copy_(torch.from_numpy(S.page_bounds(np.zeros(pg.page_bounds.shape[1:]), host(k[1])[slots], slots, ps)))
    q, kn, vn = (torch.randn(n, h, 128, device="cuda").bfloat16() for h in (8, 2, 2))
    case = (cache, pg, q, kn, vn, table, np.zeros(n, np.int64), loc)
    check_step(case, lens, "bf16", lambda: pkv.sparse_decode_step(cache, 1, pg, kn, vn, q, workspace=ws_for(n, 2, cache.max_len, ps)))


def test_step_writes_the_rows_that_it_gets_of_a_longer_slot_list():
    """out_cache_loc may be a buffer of a fixed capacity: what stands behind
    the new rows is not read."""
    rng = np.random.default_rng(47)
    lens = np.array([90, 200])
    case = step_case(rng, "bf16", 8, 2, 64, 8, lens, 6)
    cache, pg, q, kn, vn, table, rows, loc = case
    cache.out_cache_loc = dev(np.r_[loc, 10 ** 6, -5])
    pg2 = dataclasses.replace(pg, page_bounds=pg.page_bounds.clone())
    check_step(case, lens, "bf16", lambda: pkv.sparse_decode_step(cache, 1, pg, kn, vn, q, workspace=ws_for(2, 2, 200, 8)))
    pkv.page_bounds(cache, 1, pg2, n_new=2)
    clean()
    assert torch.equal(pg.page_bounds, pg2.page_bounds)


def test_step_with_nothing_to_write_and_without_entries():
    rng = np.random.default_rng(42)
    lens = np.array([90, 200])
    cache, pg, q, kn, vn, table, rows, loc = step_case(rng, "bf16", 8, 2, 64, 8, lens, 6)
    ws = ws_for(2, 2, 200, 8)
    empty = kn[:0].contiguous()
    before = cache.k_buffer.clone()
    o, sel, counts = pkv.sparse_decode_step(cache, 1, pg, empty, empty, q, workspace=ws)
    sel2, counts2 = pkv.select_pages(cache, 1, pg, q, workspace=ws)
    assert torch.equal(sel, sel2) and torch.equal(o, pkv.paged_decode_selected(cache, 1, pg, q, sel2, counts2))
    assert torch.equal(cache.k_buffer, before)
    none = dataclasses.replace(cache, req_pool_indices=cache.req_pool_indices[:0], seq_lens=cache.seq_lens[:0])
    o, sel, counts = pkv.sparse_decode_step(none, 1, pg, kn, vn, q[:0], workspace=ws)
    clean()
    assert o.shape[0] == 0 and torch.equal(cache.k_buffer[1, dev(loc).long()], kn)


def test_step_replayed_from_a_graph_and_on_other_streams():
    """Two graphs with workspaces of their own, replayed on streams of their
    own at once, and the step on a side stream, give the eager bits."""
    rng = np.random.default_rng(43)
    lens = np.array([700, 33, 1500])
    steps = []
    for i in range(2):
        case = step_case(rng, "bf16", 32, 8, 128, 16, lens, 20)
        steps.append((case, ws_for(3, 8, 1500, 16)))
    eager = [tuple(t.clone() for t in pkv.sparse_decode_step(c[0], 1, c[1], c[3], c[4], c[2], workspace=w)) for c, w in steps]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    got = pkv.sparse_decode_step(steps[0][0][0], 1, steps[0][0][1], steps[0][0][3], steps[0][0][4], steps[0][0][2], workspace=steps[0][1], stream=side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, eager[0]))
    graphs = []
    for c, w in steps:
        out = [torch.zeros_like(t) for t in eager[0]]
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            pkv.sparse_decode_step(c[0], 1, c[1], c[3], c[4], c[2], *out, workspace=w, stream=s)
        graphs.append((g, s, out))
    torch.cuda.synchronize()
    for _ in range(20):
        for g, s, _ in graphs:
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    clean()
    for (_, _, out), want in zip(graphs, eager):
        assert all(torch.equal(a, b) for a, b in zip(out, want))


@pytest.mark.parametrize("dtype,batch", [("bf16", 3), ("bf16", 90), ("f32", 5)])
def test_steps_without_a_wait_between_them(dtype, batch):
    """Each step's launches overlap the step before it: sixteen of them equal
    the four calls made one by one, bit for bit."""
    rng = np.random.default_rng(51)
    lens = rng.integers(300, 1200, batch)
    cache, pg, q, kn, vn, table, rows, loc = step_case(rng, dtype, 16, 4, 64, 4, lens, 14)
    ws = ws_for(batch, 4, 1200, 4)
    copy = dataclasses.replace(cache, k_buffer=cache.k_buffer.clone(), v_buffer=cache.v_buffer.clone())
    pg2 = dataclasses.replace(pg, page_bounds=pg.page_bounds.clone())
    steps = [tuple((torch.randn_like(x.float()) * (1 + i % 3)).to(DT[dtype]) for x in (kn, vn, q)) for i in range(16)]
    torch.cuda.synchronize()
    got = [pkv.sparse_decode_step(cache, 1, pg, *s, workspace=ws) for s in steps]
    clean()
    for (k, v, qq), (o, sel, counts) in zip(steps, got):
        pkv.kv_write(copy, 1, k, v)
        pkv.page_bounds(copy, 1, pg2)
        torch.cuda.synchronize()
        sel2, counts2 = pkv.select_pages(copy, 1, pg2, qq, workspace=ws)
        torch.cuda.synchronize()
        o2 = pkv.paged_decode_selected(copy, 1, pg2, qq, sel2, counts2)
        clean()
        assert torch.equal(sel, sel2) and torch.equal(counts, counts2) and torch.equal(o, o2)
    assert torch.equal(pg.page_bounds, pg2.page_bounds) and torch.equal(cache.k_buffer, copy.k_buffer)


def test_step_with_inputs_in_pinned_host_memory():
    rng = np.random.default_rng(44)
    lens = np.array([130, 400])
    cache, pg, q, kn, vn, table, rows, loc = step_case(rng, "bf16", 8, 2, 128, 16, lens, 9)
    ws = ws_for(2, 2, 400, 16)
    o, sel, counts = (t.clone() for t in pkv.sparse_decode_step(cache, 1, pg, kn, vn, q, workspace=ws))
    pin = [t.cpu().pin_memory() for t in (kn, vn, q, torch.zeros_like(o))]
    pkv.sparse_decode_step(cache, 1, pg, *pin[:3], o=pin[3], workspace=ws)
    torch.cuda.synchronize()
    clean()
    assert torch.equal(pin[3], o.cpu())


def test_binding_refuses_shapes_types_and_devices():
    rng = np.random.default_rng(45)
    lens = np.array([130, 400])
    cache, pg, q, kn, vn, table, rows, loc = step_case(rng, "bf16", 8, 2, 64, 16, lens, 9)
    sel, counts = pkv.select_pages(cache, 1, pg, q, workspace=ws_for(2, 2, 400, 16))
    r = dataclasses.replace
    bad = [lambda: pkv.paged_decode_selected(cache, 1, pg, q[:1], sel, counts),
           lambda: pkv.paged_decode_selected(cache, 1, pg, q, sel[:, :1].contiguous(), counts),
           lambda: pkv.paged_decode_selected(cache, 1, pg, q, sel, counts.long()),
           lambda: pkv.paged_decode_selected(cache, 1, pg, q.float(), sel, counts),
           lambda: pkv.paged_decode_selected(cache, 1, pg, q.transpose(0, 1), sel, counts),
           lambda: pkv.paged_decode_selected(cache, 1, pg, q, sel, counts, o=torch.empty_like(q)[:, :4].contiguous()),
           lambda: pkv.paged_decode_selected(cache, 1, pg, q, sel.cpu(), counts),
           lambda: pkv.select_pages(cache, 1, r(pg, page_bounds=pg.page_bounds[:, :-1].contiguous()), q),
           lambda: pkv.select_pages(cache, 1, r(pg, page_bounds=pg.page_bounds.float()), q),
           lambda: pkv.select_pages(r(cache, seq_lens=cache.seq_lens[:1]), 1, pg, q),
           lambda: pkv.select_pages(r(cache, seq_lens=None), 1, pg, q),
           lambda: pkv.sparse_decode_step(r(cache, out_cache_loc=dev(loc[:1])), 1, pg, kn, vn, q),
           lambda: pkv.page_bounds(cache, 1, pg, n_new=3),
           lambda: pkv.select_pages(cache, 1, r(pg, page_size=0), q),
           lambda: pkv.select_pages(cache, 1, pg, q[0]),
           lambda: pkv.sparse_decode_step(cache, 1, pg, kn, vn[:1].contiguous(), q),
           lambda: pkv.page_bounds(r(cache, out_cache_loc=None), 1, pg),
           lambda: pkv.page_bounds(cache, 1, r(pg, page_bounds=None))]
    for f in bad:
        with pytest.raises((ValueError, TypeError)):
            f()
    for f in (lambda: pkv.select_pages(cache, 2, pg, q), lambda: pkv.select_pages(cache, 1, r(pg, top_k=2), q, sel=sel[:, :, :2].contiguous())):
        with pytest.raises(pkv.PkvError):
            f()


def test_a_request_grows_over_pages():
    """Tables, prefill write, bounds, then steps: three requests from their
    prompts through twelve decode steps, all on tables that the GPU built,
    against the oracle at every step."""
    rng = np.random.default_rng(46)
    ps, kv, heads, d, batch, top_k = 4, 2, 8, 64, 3, 5
    lens = np.array([13, 40, 1])
    n_pages, max_pages = 64, 20
    k = torch.zeros(1, n_pages * ps, kv, d, dtype=torch.bfloat16, device="cuda")
    cache = pkv.KVCache(k_buffer=k, v_buffer=torch.zeros_like(k), req_to_token=torch.zeros(batch, max_pages * ps, dtype=torch.int32, device="cuda"),
                        req_pool_indices=dev([2, 0, 1]), seq_lens=dev(lens), out_cache_loc=torch.zeros(int(lens.sum()), dtype=torch.int32, device="cuda"), max_len=60)
    table = torch.full((batch, max_pages), -1, dtype=torch.int32, device="cuda")
    pg = pkv.SparsePages.for_cache(cache, table, ps, top_k, 1, 1)
    free, at, to = dev(rng.permutation(n_pages)), dev([0]), dev([0])
    ws = ws_for(batch, kv, 60, ps)
    pkv.build_tables(cache, table, ps, free, at, to, q_lens=dev(lens))
    kn, vn = (torch.randn(int(lens.sum()), kv, d, device="cuda").bfloat16() for _ in range(2))
    pkv.kv_write(cache, 0, kn, vn)
    pkv.page_bounds(cache, 0, pg)
    clean()
    keys, vals = [list(host(x[a:b])) for x in (kn,) for a, b in ((0, 13), (13, 53), (53, 54))], [list(host(x[a:b])) for x in (vn,) for a, b in ((0, 13), (13, 53), (53, 54))]
    cache.out_cache_loc = torch.zeros(batch, dtype=torch.int32, device="cuda")
    for _ in range(12):
        lens = lens + 1
        at, to = to, at
        cache.seq_lens = dev(lens)
        kn, vn, q = (torch.randn(batch, h, d, device="cuda").bfloat16() for h in (kv, kv, heads))
        pkv.build_tables(cache, table, ps, free, at, to)
        o, sel, counts = pkv.sparse_decode_step(cache, 0, pg, kn, vn, q, workspace=ws)
        clean()
        # the oracle holds each request's keys in order, in pages of its own
        flat_k, flat_v, tab, base = [], [], np.zeros((batch, max_pages), np.int64), 0
        for b in range(batch):
            keys[b].append(host(kn)[b])
            vals[b].append(host(vn)[b])
            n = -(-len(keys[b]) // ps)
            tab[b, :n] = base + np.arange(n)
            base += n
            pad = [np.zeros((kv, d))] * (n * ps - len(keys[b]))
            flat_k += keys[b] + pad
            flat_v += vals[b] + pad
        flat_k, flat_v = np.array(flat_k), np.array(flat_v)
        bounds = np.zeros((base, kv, 2, d))
        for b in range(batch):
            p = np.arange(lens[b])
            slots = tab[b, p // ps] * ps + p % ps
            bounds = S.page_bounds(bounds, flat_k[slots], slots, ps)
        want = S.select_pages(bounds, tab, range(batch), lens, host(q), ps, top_k, 1, 1)
        assert np.array_equal(host(sel), want[0]) and np.array_equal(host(counts), want[1])
        ref, reach = S.decode_selected(flat_k, flat_v, tab, range(batch), lens, *want, host(q), ps, d ** -0.5)
        close(o, ref, reach, flat_v, top_k * ps, "bf16")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_prompts_on_tables_from_the_gpu_with_pages_of_the_host_pool(dtype):
    """Two prompt chunks behind cached prefixes and one request without new
    tokens: tables from q_lens, the step's entries from q_lens and positions
    without a look at the host, the free list from PagePool and back to it."""
    rng = np.random.default_rng(57)
    ps, kv, heads, d, top_k, n_pages = 8, 2, 8, 64, 6, 96
    host_pool = pkv_pool.PagePool(n_pages, ps)
    old, q_lens = np.array([90, 33, 50]), np.array([40, 0, 17])
    lens, n_new = old + q_lens, int(q_lens.sum())
    rows = np.array([2, 0, 1])
    table = np.full((3, 20), -1)
    for b in range(3):
        table[rows[b], :-(-old[b] // ps)] = [host_pool.alloc() for _ in range(-(-old[b] // ps))]
    free = [host_pool.alloc() for _ in range(12)]
    k, v = pool(rng, 1, n_pages, ps, kv, d, dtype)
    ints = dict(dtype=torch.int32, device="cuda")
    cache = pkv.KVCache(k_buffer=k, v_buffer=v, req_to_token=torch.zeros(3, 20 * ps, **ints), req_pool_indices=dev(rows), seq_lens=dev(lens),
                        out_cache_loc=torch.zeros(n_new, **ints), max_len=int(lens.max()))
    pg = pkv.SparsePages.for_cache(cache, dev(table), ps, top_k, 1, 1)
    bounds = np.zeros((n_pages, kv, 2, d))
    for b in range(3):
        p = np.arange(old[b])
        slots = table[rows[b], p // ps] * ps + p % ps
        bounds = S.page_bounds(bounds, host(k)[0][slots], slots, ps)
    pg.page_bounds[0].copy_(torch.from_numpy(bounds))
    start, end, positions, ql = dev([0]), dev([0]), torch.zeros(n_new, **ints), dev(q_lens)
    kn, vn, q = (torch.randn(n_new, h, d, device="cuda").to(DT[dtype]) for h in (kv, kv, heads))
    pkv.build_tables(cache, pg.req_to_page, ps, dev(free), start, end, positions, ql)
    entry_rows = torch.repeat_interleave(cache.req_pool_indices, ql, output_size=n_new)
    step = dataclasses.replace(cache, req_pool_indices=entry_rows, seq_lens=positions + 1)
    o, sel, counts = pkv.sparse_decode_step(step, 0, pg, kn, vn, q, workspace=ws_for(n_new, kv, cache.max_len, ps))
    clean()
    want = S.build_tables(rows, lens, q_lens, table, ps, free, 0)
    assert np.array_equal(host(pg.req_to_page), want["req_to_page"])
    bounds = S.page_bounds(bounds, host(kn), want["out_cache_loc"], ps)
    assert np.array_equal(host(pg.page_bounds)[0], bounds)
    e_rows, e_lens = np.repeat(rows, q_lens), want["positions"] + 1
    chosen = S.select_pages(bounds, want["req_to_page"], e_rows, e_lens, host(q), ps, top_k, 1, 1)
    assert np.array_equal(host(sel), chosen[0]) and np.array_equal(host(counts), chosen[1])
    ref, reach = S.decode_selected(host(k)[0], host(v)[0], want["req_to_page"], e_rows, e_lens, *chosen, host(q), ps, d ** -0.5)
    close(o, ref, reach, host(v)[0], top_k * ps, dtype)
    # the requests end: their pages and the rest of the list go back
    for b in range(3):
        for page in host(pg.req_to_page)[rows[b], :-(-lens[b] // ps)]:
            host_pool.free(int(page))
    for page in free[int(end):]:
        host_pool.free(page)
    assert host_pool.num_free == n_pages
