"""Page operators and chunk attention on the GPU where a call meets bad data,
sizes at the end of 31 bits, infinities or an old workspace."""
import dataclasses

import numpy as np
import pytest
import torch

import paged_kv_cache_loc_gb300 as pkv
from paged_kv_cache_loc_gb300 import _lib
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
