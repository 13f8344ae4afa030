"""Page operators and chunk attention on the GPU where a call meets bad data,
sizes at the end of 31 bits, infinities or an old workspace."""
import dataclasses

import numpy as np
import pytest
import torch

import paged_kv_cache_loc_gb300 as pkv
from test_gpu_chunk import DTYPES, case, want
from test_gpu_chunk import host as chunk_host
from test_gpu_pages import (compact_case, dev, error, clean, gpu, host, run_compact, want_compact)  # noqa: F401 (gpu: a fixture)

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
