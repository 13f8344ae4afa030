"""The life of a cache's pages on the GPU (copy, fork, release, compact) against
its CPU oracle.  Everything here is whole numbers or copies, so all is equal,
and what a call has no business with stays as it was."""
import dataclasses

import numpy as np
import pytest
import torch

import paged_kv_cache_loc_gb300 as pkv
from oracle import pages_oracle as P
from paged_kv_cache_loc_gb300 import _lib, build

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


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).cuda()


def host(t):
    """Whole numbers, or a storage type's bits."""
    if t.is_floating_point():
        t = t.view(torch.int16 if t.dtype == torch.bfloat16 else torch.int32)
    return t.cpu().numpy()


def clean():
    status, detail = pkv.last_device_error()
    assert status == _lib.PKV_OK, detail


def error():
    status, detail = pkv.last_device_error()
    assert status == _lib.PKV_ERR_INDEX
    return detail


@dataclasses.dataclass
class Pool:
    """A pool with every element different, tables of `rows` rows, a free list."""
    cache: object
    bounds: object
    table: object
    shares: object
    free: object
    start: object
    end: object
    ps: int

    @property
    def data(self):
        return [host(x) if x is not None else None for x in (self.cache.k_buffer, self.cache.v_buffer, self.bounds)]

    def same_data(self, k, v, bounds):
        for got, want in zip(self.data, (k, v, bounds)):
            assert (got is None) == (want is None)
            if got is not None:
                assert np.array_equal(got, want)


def bits(shape, dt, seed):
    """Storage of any bit pattern, NaNs among them: copies are of bits."""
    g = torch.Generator("cuda").manual_seed(seed)
    t = torch.int16 if dt == torch.bfloat16 else torch.int32
    return torch.randint(-(1 << 15), 1 << 15, shape, generator=g, device="cuda", dtype=t).view(dt)


def pool(n_pages, ps, table, free, start, dtype="bf16", layers=2, kv=2, d=64, shares=None, bounds=True, tokens=None,
         rows=(), lens=()):
    table = np.asarray(table)
    dt = DT[dtype]
    k, v = bits((layers, n_pages * ps, kv, d), dt, 1), bits((layers, n_pages * ps, kv, d), dt, 2)
    b = bits((layers, n_pages, kv, 2, d), dt, 3) if bounds else None
    tok = torch.full((table.shape[0], table.shape[1] * ps), -3, dtype=torch.int32, device="cuda") if tokens is None else dev(tokens)
    cache = pkv.KVCache(k_buffer=k, v_buffer=v, req_to_token=tok, req_pool_indices=dev(rows), seq_lens=dev(lens))
    return Pool(cache, b, dev(table), dev(np.zeros(n_pages) if shares is None else shares), dev(free), dev([start]), dev([-9]), ps)


# ---------------------------------------------------------------------------
# copy
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("dtype,kv,d,layers", [("bf16", 8, 128, 2), ("f32", 3, 64, 1), ("bf16", 1, 8, 5), ("f32", 1, 4, 3)])
@pytest.mark.parametrize("ps", [1, 3, 16, 80])
@pytest.mark.parametrize("n", [1, 7, 40])
def test_copy_pages(dtype, kv, d, layers, ps, n):
    rng = np.random.default_rng(n + ps)
    p = pool(97, ps, np.zeros((1, 1)), [], 0, dtype, layers, kv, d, bounds=n != 7)
    perm = rng.permutation(97)
    src, dst = perm[:n].copy(), perm[n:2 * n].copy()
    if n > 7:
        src[3], src[5], src[9], dst[11] = -1, src[6], dst[9], src[11]     # passed over, a source twice, a page to itself
        src[11] = dst[11]
        src[9] = dst[9]
    want = P.copy_pages(*p.data, ps, src, dst)
    pkv.copy_pages(p.cache, ps, dev(src), dev(dst), page_bounds=p.bounds)
    clean()
    p.same_data(*want)


def test_copy_nothing_and_one_page_pools():
    p = pool(1, 4, np.zeros((1, 1)), [], 0)
    before = p.data
    pkv.copy_pages(p.cache, 4, dev([]), dev([]), page_bounds=p.bounds)
    pkv.copy_pages(p.cache, 4, dev([0, -1]), dev([0, 0]), page_bounds=p.bounds)
    clean()
    p.same_data(*before)


@pytest.mark.parametrize("src,dst", [(97, 1), (-2, 1), (1, 97), (1, -1), (2**31 - 1, 0)])
def test_copy_page_outside_the_pool(src, dst):
    p = pool(97, 16, np.zeros((1, 1)), [], 0)
    want = P.copy_pages(*p.data, 16, [5, 7], [6, 8])
    pkv.copy_pages(p.cache, 16, dev([5, src, 7]), dev([6, dst, 8]), page_bounds=p.bounds)
    assert error() == (dst if 0 <= src < 97 else src)
    p.same_data(*want)


def test_copy_on_another_stream_and_in_a_graph():
    p = pool(20, 16, np.zeros((1, 1)), [], 0, layers=4)
    src, dst = dev([1, 2]), dev([3, 4])
    want = P.copy_pages(*p.data, 16, [1, 2], [3, 4])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    pkv.copy_pages(p.cache, 16, src, dst, page_bounds=p.bounds, stream=side)
    side.synchronize()
    p.same_data(*want)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        pkv.copy_pages(p.cache, 16, src, dst, page_bounds=p.bounds)
    src.copy_(dev([5, 6]))
    dst.copy_(dev([7, 1]))
    want = P.copy_pages(*p.data, 16, [5, 6], [7, 1])
    g.replay()
    clean()
    p.same_data(*want)


# ---------------------------------------------------------------------------
# fork
# ---------------------------------------------------------------------------

def fork_case(rng, lens, fan, ps, spare=4, **kw):
    """Parents of the lengths lens (each of fan children), rows in random order."""
    lens = np.asarray(lens)
    n_par = len(lens)
    children = np.repeat(np.arange(n_par), fan)
    rows = rng.permutation(n_par + len(children) + 2)
    held = -(-lens // ps)
    width = int(held.max(initial=0)) + 2
    n_pages = int(held.sum()) + len(children) + spare
    perm = rng.permutation(n_pages)
    table = np.full((len(rows), width), -7)
    at = 0
    for i in range(n_par):
        table[rows[i], :held[i]] = perm[at:at + held[i]]
        at += held[i]
    # a child may take over less than the parent holds
    take = np.array([rng.integers(0, n + 1) if c % 3 == 2 else n for c, n in enumerate(np.repeat(lens, fan))])
    order = rng.permutation(len(children))
    shares = np.zeros(n_pages, np.int64)
    shares[perm[:at // 3]] = 2
    p = pool(n_pages, ps, table, np.r_[[-5, -5], perm[at:]], 2, shares=shares, rows=rows[n_par:n_par + len(children)],
             lens=take[order], **kw)
    return p, rows[:n_par][children[order]]


def run_fork(p, parents, token_table=True, **kw):
    pkv.fork_requests(p.cache, p.table, p.ps, dev(parents), p.shares, p.free, p.start, p.end, page_bounds=p.bounds,
                      token_table=token_table, **kw)


def want_fork(p, parents, token_table=True):
    return P.fork(*p.data, p.ps, host(p.table), host(p.cache.req_to_token) if token_table else None, host(p.shares),
                  host(p.cache.req_pool_indices), parents, host(p.cache.seq_lens), host(p.free), int(p.start))


def check_fork(p, want):
    k, v, b, table, tokens, shares, end = want
    p.same_data(k, v, b)
    assert np.array_equal(host(p.table), table)
    assert np.array_equal(host(p.shares), shares)
    assert int(p.end) == end
    if tokens is not None:
        assert np.array_equal(host(p.cache.req_to_token), tokens)
    else:
        assert (host(p.cache.req_to_token) == -3).all()


@pytest.mark.parametrize("ps", [1, 3, 16, 64])
@pytest.mark.parametrize("lens,fan", [([1], 1), ([0], 3), ([15, 16, 17], 2), ([128, 0, 100, 1, 64, 63, 65], 3), ([700], 8),
                                      (list(range(40)), 10)])
@pytest.mark.parametrize("dtype,extras", [("bf16", True), ("f32", False)])
def test_fork(ps, lens, fan, dtype, extras):
    rng = np.random.default_rng(ps + len(lens))
    p, parents = fork_case(rng, lens, fan, ps, dtype=dtype, bounds=extras, layers=3)
    want = want_fork(p, parents, extras)
    run_fork(p, parents, token_table=extras)
    clean()
    check_fork(p, want)


def test_fork_a_whole_models_layers():
    rng = np.random.default_rng(8)
    p, parents = fork_case(rng, [1003], 8, 16, layers=32, kv=8, d=128)
    want = want_fork(p, parents)
    run_fork(p, parents)
    clean()
    check_fork(p, want)


def test_fork_no_entries():
    p = pool(4, 16, np.zeros((2, 2)), [1, 2], 1)
    before = p.data
    run_fork(p, [])
    clean()
    p.same_data(*before)
    assert int(p.end) == 1


def test_fork_free_list_runs_out():
    """Entries behind the list's end get -1; those before it are exact."""
    rng = np.random.default_rng(3)
    p, parents = fork_case(rng, [5, 6, 7], 1, 16)
    p.cache.seq_lens.copy_(dev([5, 5, 5]))
    p.free = p.free[:4].clone()                         # two pages
    want = want_fork(dataclasses.replace(p, free=torch.cat([p.free, p.free[2:3]])), parents)
    run_fork(p, parents)
    assert error() == -300002
    rows = host(p.cache.req_pool_indices)
    assert host(p.table)[rows[2], 0] == -1 and (host(p.cache.req_to_token)[rows[2], :5] == -1).all()
    assert int(p.end) == 4
    assert np.array_equal(np.delete(host(p.table), rows[2], 0), np.delete(want[3], rows[2], 0))


@pytest.mark.parametrize("what,value,detail", [("child", 99, 99), ("child", -1, -1), ("parent", 77, 77), ("len", -1, -1),
                                               ("len", 10**6, 10**6), ("itself", 0, None)])
def test_fork_bad_entry_counts_as_empty(what, value, detail):
    rng = np.random.default_rng(4)
    p, parents = fork_case(rng, [20, 40], 2, 16)
    parents = parents.copy()
    rows, lens = host(p.cache.req_pool_indices).copy(), host(p.cache.seq_lens).copy()
    lens[:] = 20
    p.cache.seq_lens.copy_(dev(lens))
    good = lens.copy()
    good[1] = 0
    want = want_fork(dataclasses.replace(p, cache=dataclasses.replace(p.cache, seq_lens=dev(good))), parents)
    if what == "child":
        rows[1] = value
    elif what == "parent":
        parents[1] = value
    elif what == "len":
        lens[1] = value
    else:
        parents[1] = rows[1]
        detail = rows[1]
    p.cache.req_pool_indices.copy_(dev(rows))
    p.cache.seq_lens.copy_(dev(lens))
    run_fork(p, parents)
    assert error() == detail
    check_fork(p, want)


def test_fork_bad_page_of_the_parent():
    rng = np.random.default_rng(4)
    p, parents = fork_case(rng, [40], 1, 16, bounds=False)
    row, child = int(parents[0]), int(host(p.cache.req_pool_indices)[0])
    p.cache.seq_lens.copy_(dev([40]))
    p.table[row, 1] = 10**6
    want = want_fork(dataclasses.replace(p, cache=dataclasses.replace(p.cache, seq_lens=dev([16]))), parents)[5]
    run_fork(p, parents)
    assert error() == 10**6
    got = host(p.table)[child]
    assert got[0] == host(p.table)[row, 0] and got[1] == -1 and got[2] == host(p.free)[2]
    assert np.array_equal(host(p.shares), want)
    tok = host(p.cache.req_to_token)[child]
    assert (tok[16:32] == -1).all() and (tok[32:40] == got[2] * 16 + np.arange(8)).all()


# ---------------------------------------------------------------------------
# release
# ---------------------------------------------------------------------------

def release_case(rng, lens, ps, shared=0.5, width=0, rows_more=2):
    """Rows of the lengths lens; a part of the pages belongs to the next row too."""
    lens = np.asarray(lens)
    b = len(lens)
    held = -(-lens // ps)
    width = max(width, int(held.max(initial=0)) + 1)
    rows = rng.permutation(b + rows_more)
    table = np.full((b + rows_more, width), -1)
    n_pages = int(held.sum()) + 9
    perm = rng.permutation(n_pages)
    at = 0
    for i in range(b):
        common = int(min(held[i], held[i - 1]) * shared) if i % 4 else 0
        table[rows[i], :common] = table[rows[i - 1], :common]
        m = held[i] - common
        table[rows[i], common:held[i]] = perm[at:at + m]
        at += m
    count = np.zeros(n_pages, np.int64)
    np.add.at(count, table[table >= 0], 1)
    return pool(n_pages, ps, table, np.r_[np.full(at, -5), perm[at:]], at, layers=1, kv=1, d=8, shares=np.maximum(count - 1, 0),
                bounds=False, rows=rows[:b], lens=lens)


def run_release(p, keep=None, **kw):
    pkv.release_pages(p.cache, p.table, p.ps, p.shares, p.free, p.start, p.end, keep, **kw)


def check_release(p, want):
    table, shares, free, end = want
    assert np.array_equal(host(p.table), table)
    assert np.array_equal(host(p.shares), shares)
    assert np.array_equal(host(p.free), free)
    assert int(p.end) == end


def want_release(p, keep=None):
    lens = host(p.cache.seq_lens)
    return P.release(host(p.table), host(p.shares), p.ps, host(p.cache.req_pool_indices), lens,
                     np.zeros_like(lens) if keep is None else keep, host(p.free), int(p.start))


@pytest.mark.parametrize("ps", [1, 3, 16])
@pytest.mark.parametrize("lens", [[0], [1], [17, 16, 15], [300, 0, 1, 100, 200], list(range(0, 700, 3)), [5000]])
@pytest.mark.parametrize("kept", [False, True])
@pytest.mark.parametrize("width", [0, 20000])         # the wide table takes the launch of two kernels
def test_release(ps, lens, kept, width):
    rng = np.random.default_rng(len(lens) + ps)
    p = release_case(rng, lens, ps, width=width)
    keep = np.array([rng.integers(0, n + 1) for n in lens]) if kept else None
    want = want_release(p, keep)
    run_release(p, None if keep is None else dev(keep))
    clean()
    check_release(p, want)


def test_release_a_large_pool():
    """More pages than one round of the cluster's warps, most of them freed."""
    rng = np.random.default_rng(2)
    p = release_case(rng, rng.integers(1, 3000, 400), 1)
    assert p.shares.numel() > 1 << 18
    want = want_release(p)
    run_release(p)
    clean()
    check_release(p, want)


def test_release_nothing():
    p = release_case(np.random.default_rng(0), [40, 50], 16)
    want = want_release(p, [40, 50])
    run_release(p, dev([40, 50]))
    clean()
    check_release(p, want)
    empty = dataclasses.replace(p, cache=dataclasses.replace(p.cache, req_pool_indices=dev([]), seq_lens=dev([])))
    run_release(empty)
    clean()
    assert int(p.end) == int(p.start)


@pytest.mark.parametrize("width", [0, 40000])
def test_release_a_row_named_twice(width):
    """Its pages are given back once."""
    p = release_case(np.random.default_rng(1), [100, 60], 16, shared=0, width=width)
    want = want_release(p)
    rows = host(p.cache.req_pool_indices)
    p.cache.req_pool_indices, p.cache.seq_lens = dev([rows[0], rows[1], rows[0]]), dev([100, 60, 100])
    run_release(p)
    assert error() == -1
    check_release(p, want)


def test_release_more_references_than_a_page_has():
    p = release_case(np.random.default_rng(1), [32, 32], 16, shared=0)
    rows = host(p.cache.req_pool_indices)
    p.table[rows[1], 1] = p.table[rows[0], 0]             # held twice, counted once
    pages = sorted({*host(p.table)[rows].flatten().tolist()} - {-1})
    first = int(p.table[rows[0], 0])
    run_release(p)
    assert error() == -400000 - int(host(p.free)[int(p.end):int(p.start)][pages.index(first)])
    assert int(p.end) == int(p.start) - 3
    assert host(p.free)[int(p.end):int(p.start)].tolist() == pages
    assert (host(p.shares) == 0).all()


@pytest.mark.parametrize("what,value", [("row", 55), ("row", -1), ("len", -4), ("len", 10**7), ("keep", 101), ("keep", -1)])
def test_release_bad_entry_gives_nothing(what, value):
    p = release_case(np.random.default_rng(5), [100, 100, 100], 16, shared=0)
    rows, lens, keep = host(p.cache.req_pool_indices).copy(), np.array([100] * 3), np.array([10] * 3)
    want = want_release(p, np.array([10, 100, 10]))
    {"row": rows, "len": lens, "keep": keep}[what][1] = value
    p.cache.req_pool_indices, p.cache.seq_lens = dev(rows), dev(lens)
    run_release(p, dev(keep))
    assert error() == value
    check_release(p, want)


def test_release_more_than_the_list_has_room_for():
    p = release_case(np.random.default_rng(6), [100], 16, shared=0)
    pages = np.sort(host(p.table)[host(p.cache.req_pool_indices)[0], :7])
    tail = host(p.free)[3:]
    p.start = dev([3])
    run_release(p)
    assert error() == 7
    assert int(p.end) == 0
    assert host(p.free)[:3].tolist() == pages[4:].tolist() and np.array_equal(host(p.free)[3:], tail)


# ---------------------------------------------------------------------------
# compact
# ---------------------------------------------------------------------------

def compact_case(rng, n_pages, n_free, ps=4, rows=6, skip=3, **kw):
    perm = rng.permutation(n_pages)
    free, used = perm[:n_free], perm[n_free:]
    width = -(-max(1, len(used)) // rows) + 1
    table = np.full((rows, width), -1)
    for i, p in enumerate(used):
        table[i % rows, i // rows] = p
    if rows > 1 and len(used) >= rows:
        table[0, 0] = table[1, 0]                             # a shared page; another belongs to no row
    table[-1, -1] = free[0] if n_free else -9                 # what is left of an old entry
    shares = np.zeros(n_pages, np.int64)
    shares[used] = rng.integers(0, 5, len(used))
    tokens = np.where(table[:, :, None] >= 0, table[:, :, None] * ps + np.arange(ps), -1).reshape(rows, -1)
    return pool(n_pages, ps, table, np.r_[np.full(skip, 1), free], skip, shares=shares, tokens=tokens, **kw)


def run_compact(p, token_table=True, ws=None, **kw):
    ws = ws or pkv.compact_workspace(p.shares.numel())
    return pkv.compact_pages(p.cache, p.table, p.ps, p.shares, p.free, p.start, page_bounds=p.bounds, token_table=token_table,
                             workspace=ws, **kw)


def want_compact(p, token_table=True):
    return P.compact(*p.data, p.ps, host(p.table), host(p.cache.req_to_token) if token_table else None, host(p.shares), host(p.free),
                     int(p.start))


def check_compact(p, want, remap, free=None):
    k, v, b, table, tokens, shares, listed, to = want
    p.same_data(k, v, b)
    assert np.array_equal(host(p.table), table)
    if tokens is not None:
        assert np.array_equal(host(p.cache.req_to_token), tokens)
    assert np.array_equal(host(p.shares), shares)
    assert np.array_equal(host(p.free if free is None else free), listed)
    assert np.array_equal(host(remap), to)


@pytest.mark.parametrize("n_pages,n_free", [(1, 0), (1, 1), (2, 1), (7, 3), (64, 0), (64, 64), (128, 1), (129, 128), (300, 150),
                                            (1000, 900), (1000, 70), (40000, 20000)])
@pytest.mark.parametrize("dtype,extras", [("bf16", True), ("f32", False)])
def test_compact(n_pages, n_free, dtype, extras):
    rng = np.random.default_rng(n_pages + n_free)
    p = compact_case(rng, n_pages, n_free, dtype=dtype, bounds=extras, kv=1, d=8, layers=3)
    before = host(p.cache.req_to_token)
    want = want_compact(p, extras)
    remap = run_compact(p, token_table=extras)
    clean()
    check_compact(p, want, remap)
    if not extras:
        assert np.array_equal(host(p.cache.req_to_token), before)
    # a pool that is compact stays as it is
    want = want_compact(p, extras)
    check_compact(p, want, run_compact(p, token_table=extras))
    assert (host(p.free)[3:] == np.arange(n_pages - n_free, n_pages)).all()


def test_compact_into_another_list_and_pages_of_many_pieces():
    rng = np.random.default_rng(9)
    p = compact_case(rng, 30, 14, ps=80, kv=8, d=128)
    want, free, out = want_compact(p), host(p.free), p.free.clone()
    remap = torch.full((30,), -7, dtype=torch.int32, device="cuda")
    got = run_compact(p, free_out=out, remap=remap)
    clean()
    assert got is remap
    check_compact(p, want, remap, out)
    assert np.array_equal(host(p.free), free)


@pytest.mark.parametrize("value", [64, -1, "twice"])
def test_compact_bad_free_list(value):
    """The page that is named twice, or none at all, is an error; nothing faults."""
    p = compact_case(np.random.default_rng(2), 64, 20)
    p.free[7] = int(p.free[8]) if value == "twice" else value
    detail = int(p.free[7])
    run_compact(p)
    assert error() == detail


def test_compact_refusals():
    p = compact_case(np.random.default_rng(2), 640, 20)
    for ws, status in ((None, _lib.PKV_ERR_WORKSPACE), (pkv.compact_workspace(64), _lib.PKV_ERR_WORKSPACE)):
        with pytest.raises(pkv.PkvError) as e:
            pkv.compact_pages(p.cache, p.table, p.ps, p.shares, p.free, p.start, workspace=ws)
        assert e.value.status == status
    clean()


@pytest.mark.parametrize("what", ["compact", "release"])
def test_calls_of_two_kernels_in_a_graph(what):
    """Replayed on other counts and tables than those of the capture."""
    rng = np.random.default_rng(4)
    if what == "compact":
        p = compact_case(rng, 700, 300)
        ws, out = pkv.compact_workspace(700), p.free.clone()
        remap = torch.zeros(700, dtype=torch.int32, device="cuda")
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            run_compact(p, ws=ws, free_out=out, remap=remap)
        other = compact_case(np.random.default_rng(5), 700, 300)
        for mine, theirs in ((p.table, other.table), (p.shares, other.shares), (p.free, other.free),
                             (p.cache.req_to_token, other.cache.req_to_token)):
            mine.copy_(theirs)
        out.copy_(p.free)
        want = want_compact(p)
        g.replay()
        clean()
        check_compact(p, want, remap, out)
    else:
        p = release_case(rng, [300, 5, 77, 1000], 3, width=20000)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            run_release(p)
        other = release_case(np.random.default_rng(6), [300, 5, 77, 1000], 3, width=20000)
        for mine, theirs in ((p.table, other.table), (p.shares, other.shares), (p.free, other.free), (p.start, other.start),
                             (p.cache.req_pool_indices, other.cache.req_pool_indices)):
            mine.copy_(theirs)
        want = want_release(p)
        g.replay()
        clean()
        check_release(p, want)


def test_two_streams():
    """Two pools at once, each on a stream of its own."""
    rng = np.random.default_rng(14)
    a, b = (release_case(rng, rng.integers(1, 400, 100), 2) for _ in range(2))
    want = [want_release(a), want_release(b)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    for p, s in zip((a, b), streams):
        run_release(p, stream=s)
    torch.cuda.synchronize()
    clean()
    for p, w in zip((a, b), want):
        check_release(p, w)


# ---------------------------------------------------------------------------
# refusals of the binding, and a run of them together
# ---------------------------------------------------------------------------

def test_refusals():
    p = pool(8, 16, np.zeros((2, 4)), [1, 2, 3], 0, rows=[0], lens=[5])
    ints = dev([0])
    with pytest.raises(ValueError, match="page_size"):
        pkv.copy_pages(p.cache, 0, ints, ints)
    with pytest.raises(ValueError, match="dst must have 1"):
        pkv.copy_pages(p.cache, 16, ints, dev([0, 1]))
    with pytest.raises(TypeError, match="src"):
        pkv.copy_pages(p.cache, 16, ints.long(), ints)
    with pytest.raises(ValueError, match="page_bounds"):
        pkv.copy_pages(p.cache, 16, ints, ints, page_bounds=p.bounds[:1])
    with pytest.raises(ValueError, match="pinned"):
        pkv.copy_pages(p.cache, 16, ints.cpu(), ints)
    with pytest.raises(ValueError, match="contiguous"):
        pkv.copy_pages(p.cache, 16, dev([1, 2, 3, 4])[::2], dev([5, 6]))
    with pytest.raises(pkv.PkvError):                       # 128 slots are no whole number of pages of 24
        pkv.copy_pages(p.cache, 24, ints, ints)
    with pytest.raises(ValueError, match="parents must have 1"):
        run_fork(p, [0, 1])
    with pytest.raises(ValueError, match="shares must have 8"):
        run_fork(dataclasses.replace(p, shares=p.shares[:5].contiguous()), [1])
    with pytest.raises(ValueError, match="req_to_token"):
        run_fork(dataclasses.replace(p, cache=dataclasses.replace(p.cache, req_to_token=p.cache.req_to_token[:1])), [1])
    with pytest.raises(pkv.PkvError):                       # the list's new place is a word of its own
        run_fork(dataclasses.replace(p, end=p.start), [1])
    with pytest.raises(pkv.PkvError):
        run_release(dataclasses.replace(p, end=p.start))
    with pytest.raises(ValueError, match="seq_lens"):
        run_release(dataclasses.replace(p, cache=dataclasses.replace(p.cache, seq_lens=None)))
    with pytest.raises(ValueError, match="keep_lens must have 1"):
        run_release(p, dev([0, 0]))
    with pytest.raises(ValueError, match="remap must have 8"):
        run_compact(p, remap=dev([0, 1]))
    with pytest.raises(ValueError, match="free_out must have 3"):
        run_compact(p, free_out=dev([0, 1]))
    clean()


def test_a_life_of_pages_in_a_graph():
    """Four rounds of one captured loop: a request is forked into two samples,
    each gets a token's page from build_tables, the samples are given back, and
    the list ends with the pages it began with."""
    rng = np.random.default_rng(12)
    ps, n_pages = 4, 40
    p = pool(n_pages, ps, np.full((4, 8), -1), rng.permutation(n_pages), 0, kv=1, d=8, rows=[1], lens=[10])
    i32 = dict(dtype=torch.int32, device="cuda")
    c = dataclasses.replace(p.cache, out_cache_loc=torch.full((10,), -1, **i32))
    pkv.build_tables(c, p.table, ps, p.free, p.start, p.end, q_lens=dev([10]))
    two = dataclasses.replace(p.cache, req_pool_indices=dev([0, 3]), seq_lens=dev([10, 10]))
    grown = dataclasses.replace(two, seq_lens=dev([13, 13]), out_cache_loc=torch.full((6,), -1, **i32))
    mid, top, back = (torch.zeros(1, **i32) for _ in range(3))
    first = host(p.free)
    q = dev([3, 3])

    def loop():
        pkv.fork_requests(two, p.table, ps, dev_parents, p.shares, p.free, p.end, mid, page_bounds=p.bounds)
        pkv.build_tables(grown, p.table, ps, p.free, mid, top, q_lens=q)
        loc.copy_(grown.out_cache_loc)
        pkv.release_pages(grown, p.table, ps, p.shares, p.free, top, back)

    dev_parents, loc = dev([1, 1]), torch.zeros(6, **i32)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        loop()
    for _ in range(4):
        g.replay()
        clean()
        assert int(p.end) == 3 and int(mid) == 5 and int(top) == 7 and int(back) == 3
        assert sorted(host(p.free)[3:]) == sorted(first[3:]) and (host(p.shares) == 0).all()
        assert (host(loc) >= 0).all() and len(set(host(loc).tolist())) == 6
        t = host(p.table)
        assert (t[[0, 3], :4] == -1).all() and t[1, 0] >= 0
