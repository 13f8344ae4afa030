"""Page operators and chunk attention on the GPU where a call meets bad data,
sizes at the end of 31 bits, infinities or an old workspace."""
import dataclasses

import numpy as np
import pytest
import torch

import paged_kv_cache_loc_gb300 as pkv
from test_gpu_chunk import DTYPES, case, check, want
from test_gpu_chunk import host as chunk_host
from test_gpu_pages import (clean, compact_case, dev, error, fork_case, gpu, host, run_compact, run_fork,  # noqa: F401 (gpu: a fixture)
                            want_compact)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("value", [64, -1, 2**31 - 1, "twice"])
@pytest.mark.parametrize("in_place", [True, False])
def test_compact_bad_free_list_names_no_used_page(value, in_place):
    """The free pages are those that the list names; what is left of it is -1,
    so that who takes from it later gets no page that a row holds."""
    p = compact_case(np.random.default_rng(2), 64, 20)
    p.table[-1, -1] = -9                                      # (else what is left of an old entry)
    p.free[7] = int(p.free[8]) if value == "twice" else value
    detail = int(p.free[7])
    want, out = want_compact(p), p.free.clone()
    remap = run_compact(p, free_out=None if in_place else out)
    assert error() == detail
    k, v, b, table, tokens, shares, _, to = want
    p.same_data(k, v, b)
    assert np.array_equal(host(p.table), table) and np.array_equal(host(p.cache.req_to_token), tokens)
    assert np.array_equal(host(p.shares), shares) and np.array_equal(host(remap), to)
    listed = host(p.free if in_place else out)
    assert listed[:3].tolist() == [1, 1, 1] and listed[3:].tolist() == [*range(45, 64), -1]
    # twenty rows that each need a page: the last gets none
    children = dataclasses.replace(p.cache, req_pool_indices=dev(range(1, 21)), seq_lens=dev([1] * 20), req_to_token=dev(np.full((21, 4), -1)))
    rows, end = dev(np.full((21, 1), -1)), dev([0])
    rows[0, 0] = 0
    pkv.fork_requests(children, rows, p.ps, dev([0] * 20), p.shares, dev(listed), p.start, end)
    assert error() == -1
    taken = host(rows)[1:, 0].tolist()
    assert taken == [*range(45, 64), -1] and not set(taken[:19]) & set(table[table >= 0].tolist())


# ---------------------------------------------------------------------------
# rows of 2^31 - 1 positions: the step behind the last one passes 31 bits
# ---------------------------------------------------------------------------

TOP = 2**31 - 1


def room(n_bytes):
    torch.cuda.empty_cache()
    if torch.cuda.mem_get_info()[0] < n_bytes + (8 << 30):
        pytest.skip("not enough free memory")


def small_pool(pages, layers=1, kv=1, d=8, dtype=torch.bfloat16):
    return [torch.zeros(layers, pages, kv, d, dtype=dtype, device="cuda") for _ in range(2)]


def test_release_the_end_of_a_row_of_two_billion_pages():
    room(4 * TOP)
    i32, n = dict(dtype=torch.int32, device="cuda"), 5000
    k, v = small_pool(n)
    table = torch.empty(1, TOP, **i32)
    pages = dev(np.random.default_rng(0).permutation(n))
    table[0, TOP - n - 99:TOP - n] = 7
    table[0, TOP - n:] = pages
    cache = pkv.KVCache(k_buffer=k, v_buffer=v, req_to_token=table, req_pool_indices=dev([0]), seq_lens=dev([TOP]))
    shares, free, end = torch.zeros(n, **i32), torch.full((n,), -5, **i32), dev([-1])
    shares[:100] = 3
    pkv.release_pages(cache, table, 1, shares, free, dev([n]), end, dev([TOP - n]))
    clean()
    assert (table[0, TOP - n:] == -1).all() and (table[0, TOP - n - 99:TOP - n] == 7).all()
    assert host(shares).tolist() == [2] * 100 + [0] * (n - 100)
    assert int(end) == 100 and host(free).tolist() == [-5] * 100 + list(range(100, n))


def test_fork_a_row_of_two_billion_positions():
    room(6 * 4 * TOP)
    i32, n = dict(dtype=torch.int32, device="cuda"), 64
    k, v = small_pool(n, layers=32, kv=64, d=128, dtype=torch.float32)      # (a page of many pieces: many CTAs to the child)
    table, tokens = torch.empty(2, TOP, **i32), torch.empty(2, TOP, **i32)
    torch.arange(TOP, out=table[1])
    table[1] %= n
    table[0].fill_(-7)
    tokens.fill_(-3)
    cache = pkv.KVCache(k_buffer=k, v_buffer=v, req_to_token=tokens, req_pool_indices=dev([0]), seq_lens=dev([TOP]))
    shares, end = torch.zeros(n, **i32), dev([-1])
    pkv.fork_requests(cache, table, 1, dev([1]), shares, dev([]), dev([0]), end)
    clean()
    assert torch.equal(table[0], table[1]) and torch.equal(tokens[0], table[1])
    assert (tokens[1] == -3).all() and int(end) == 0
    assert host(shares).tolist() == [TOP // n + (p < TOP % n) for p in range(n)]


# ---------------------------------------------------------------------------
# chunk attention: scores of -inf
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("G,q_lens,lens", [(1, [5, 2], [3, 40]), (4, [5, 2], [2000, 40]), (1, [300, 2], [200, 40]), (8, [40, 3], [4500, 40]),
                                           (2, [400, 70], [520, 300])])
def test_scores_of_minus_infinity(dtype, causal, d, G, q_lens, lens):
    """Entry 0, kv head 0: a row whose scores are all -inf gives NaN (0 / 0), one
    that sees nothing 0, and with one finite score its value alone, exactly."""
    c = case(q_lens, lens, dtype=dtype, G=G, d=d, kv=2, ps=16)
    c.q[..., 0] = c.q[..., 0].abs() + 0.5
    ref, tol = want(c, causal)
    n, q = lens[0], q_lens[0]
    pos = np.arange(n)
    slots = torch.from_numpy(chunk_host(c.table)[int(c.cache.req_pool_indices[0]), pos // 16] * 16 + pos % 16).cuda()
    sees = np.arange(q) + n - q >= 0 if causal else np.ones(q, bool)
    k, v = c.cache.k_buffer, c.cache.v_buffer
    first = k[0, slots[0], 0].clone()
    k[0, slots, 0, 0] = -float("inf")
    for ws in (None, c.workspace()):
        got = chunk_host(c.run(causal, workspace=ws))
        assert np.isnan(got[:q, :G][sees]).all() and (got[:q, :G][~sees] == 0).all()
        rest = np.ones(got.shape, bool)
        rest[:q, :G] = False
        assert (np.abs(got - ref) <= tol)[rest].all()
    k[0, slots[0], 0] = first
    alone = chunk_host(v[0, slots[0], 0])
    for ws in (None, c.workspace()):
        got = chunk_host(c.run(causal, workspace=ws))
        assert (got[:q, :G][sees] == alone).all() and (got[:q, :G][~sees] == 0).all()
        assert (np.abs(got - ref) <= tol)[rest].all()
    clean()


# ---------------------------------------------------------------------------
# chunk attention: moved pages, values that are not finite, old workspaces
# ---------------------------------------------------------------------------

KINDS = [([5, 1], [700, 90]), ([8, 3], [4500, 1300]), ([300, 70], [900, 200]), ([40, 2], [4500, 64])]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("ps", [3, 16])
@pytest.mark.parametrize("q_lens,lens", KINDS)
def test_moving_pages_changes_no_bit(dtype, d, ps, q_lens, lens):
    """The same calls before and after the pool is compacted, alone and together,
    with a workspace and without."""
    c = case(q_lens, lens, dtype=dtype, d=d, G=8, ps=ps, kv=1, spare_pages=300)
    entries = [dataclasses.replace(c, q=c.q[lo:hi].contiguous(), max_q=hi - lo, cache=dataclasses.replace(
        c.cache, req_pool_indices=c.cache.req_pool_indices[i:i + 1].clone(), seq_lens=c.cache.seq_lens[i:i + 1].clone(), max_len=lens[i],
        qo_indptr=dev([0, hi - lo]))) for i, (lo, hi) in enumerate(((0, q_lens[0]), (q_lens[0], sum(q_lens))))]
    calls = [(x, ws) for x in [c, *entries] for ws in (None, x.workspace())]
    before = [x.run(workspace=ws).clone() for x, ws in calls]
    n_pages = c.cache.k_buffer.shape[1] // ps
    held = set(chunk_host(c.table).flatten().tolist()) - {-1}
    free = dev([p for p in np.random.default_rng(1).permutation(n_pages) if p not in held])
    remap = pkv.compact_pages(c.cache, c.table, ps, dev(np.zeros(n_pages)), free, dev([0]), token_table=False,
                              workspace=pkv.compact_workspace(n_pages))
    assert int((remap != torch.arange(n_pages, device="cuda")).sum()) > 10 and int(c.table.max()) == len(held) - 1
    for (x, ws), o in zip(calls, before):
        assert torch.equal(x.run(workspace=ws), o)
    clean()


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("G,q_lens,lens", [(1, [600, 3], [4200, 10]), (2, [300, 3], [4200, 10]), (1, [128, 3], [4200, 10]), (8, [16, 3], [4200, 10])])
def test_values_that_some_rows_see(dtype, d, bad, G, q_lens, lens):
    """One value that is not finite, at places of the causal diagonal, before it
    and behind tiles' borders: the rows that see it have their channel not
    finite, everything else is as without it."""
    c = case(q_lens, lens, dtype=dtype, d=d, G=G, kv=2, ps=8)
    ref, tol = want(c)
    n, q = lens[0], q_lens[0]
    row = int(c.cache.req_pool_indices[0])
    lim = np.r_[n - q + np.arange(q), np.full(q_lens[1], -1)]
    for ws in (None, c.workspace()):
        for j in {100, n - q, n - q + 1, n - q // 2, (n - 1) // 128 * 128, (n - 1) // 128 * 128 - 1, n - 1}:
            slot = int(c.table[row, j // 8]) * 8 + j % 8
            keep = c.cache.v_buffer[0, slot, 1, 7].clone()
            c.cache.v_buffer[0, slot, 1, 7] = bad
            got, sees = chunk_host(c.run(workspace=ws)), lim >= j
            c.cache.v_buffer[0, slot, 1, 7] = keep
            assert not np.isfinite(got[sees][:, G:, 7]).any(), j
            rest = np.ones_like(got, bool)
            rest[sees, G:, 7] = False
            assert (np.abs(got - ref) <= tol)[rest].all(), j
    clean()


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("q_lens,lens", KINDS + [([2] * 40, [0, 1, 130, 2000] * 10)])
def test_a_workspace_of_anything(dtype, d, q_lens, lens):
    """What an earlier call, or nobody, left in the workspace does not matter, a
    call repeats itself bit for bit, and nothing is written behind its bytes."""
    c = case(q_lens, lens, dtype=dtype, d=d, G=8, kv=1, ps=16)
    ref, tol = want(c)
    ws = c.workspace()
    start = ws.desc.base - ws.buffer.data_ptr()
    end = start + ws.desc.bytes
    outside = torch.cat([ws.buffer[:start], ws.buffer[end:]]).fill_(0xA5)
    ws.buffer[:start], ws.buffer[end:] = 0xA5, 0xA5
    first = None
    for fill in (0x00, 0xFF, 0x7F, None, 0x01):
        if fill is None:
            other = case([1, 7, 3], [64, 3000, 500], dtype=dtype, d=d, G=8, kv=1, ps=16)
            other.run(workspace=ws)
        else:
            ws.buffer[start:end] = fill
        o = torch.full_like(c.q, float("nan"))
        c.run(o=o, workspace=ws)
        first = o if first is None else first
        assert torch.equal(o, first)
        assert torch.equal(torch.cat([ws.buffer[:start], ws.buffer[end:]]), outside)
    check(first, ref, tol)
    clean()


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("q_lens,lens", KINDS)
def test_rows_before_the_first_entry_stay(dtype, q_lens, lens):
    c = case(q_lens, lens, dtype=dtype, spare_rows=20)
    c.cache.qo_indptr += 13
    o = torch.full_like(c.q, 3.25)
    ref, tol = want(c, o=o)
    for ws in (None, c.workspace()):
        o.fill_(3.25)
        check(c.run(o=o, workspace=ws), ref, tol)
        assert (o[:13] == 3.25).all() and (o[13 + sum(q_lens):] == 3.25).all()
    clean()


def test_fork_bad_last_page_of_the_parent():
    """The child has a page of its own where the parent's partly filled one is
    none of the pool's, without a copy: nothing of another page is written."""
    p, parents = fork_case(np.random.default_rng(4), [40], 1, 16)
    row, child = int(parents[0]), int(host(p.cache.req_pool_indices)[0])
    p.cache.seq_lens.copy_(dev([40]))
    p.table[row, 2] = -4
    before, taken = p.data, int(p.free[2])
    run_fork(p, parents)
    assert error() == -4
    assert host(p.table)[child, :3].tolist() == [*host(p.table)[row, :2].tolist(), taken] and int(p.end) == 3
    p.same_data(*before)


def test_fork_a_place_outside_the_list():
    """No page is taken: the entries' partly filled pages are -1."""
    for start in (-1, 10**6):
        p, parents = fork_case(np.random.default_rng(4), [40, 32], 1, 16)
        p.cache.seq_lens.copy_(dev([40, 32]))
        order = host(p.cache.req_pool_indices)
        p.start = dev([start])
        before = p.data
        run_fork(p, parents)
        assert error() == start and int(p.end) == p.free.numel()
        assert host(p.table)[order[0], 2] == -1
        p.same_data(*before)
