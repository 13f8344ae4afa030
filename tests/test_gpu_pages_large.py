"""Copies, forks and chunk attention with rows more than 4 GB past the pool's
base: a 32-bit offset would wrap onto the first layer's first rows."""
import numpy as np
import pytest
import torch

import paged_kv_cache_loc_gb300 as pkv
from oracle import pages_oracle as P
from paged_kv_cache_loc_gb300 import _lib, build
from test_gpu_chunk import Case, check, dev, host

pytestmark = pytest.mark.gpu

BASE, PAGE, TAIL = 1 << 20, 16, 64             # slots before the case's pages; pages behind them


@pytest.fixture(scope="module", autouse=True)
def gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    build.build()
    torch.cuda.set_device(0)
    pkv.last_device_error()


def big(dtype, d, kv):
    size = BASE + TAIL * PAGE
    k, v = (torch.empty(2, size, kv, d, dtype=dtype, device="cuda") for _ in range(2))
    assert size * kv * d * k.element_size() >= 1 << 31
    g = torch.Generator("cuda").manual_seed(3)
    for x in (k, v):
        x[:, :2 * TAIL * PAGE] = 0
        x[:, BASE:] = torch.randn(2, TAIL * PAGE, kv, d, generator=g, device="cuda").to(dtype)
    return k, v


@pytest.mark.parametrize("dtype,d,kv", [(torch.bfloat16, 128, 8), (torch.float32, 128, 4)])
def test_copy_fork_and_chunk_far_behind(dtype, d, kv):
    k, v = big(dtype, d, kv)
    first = BASE // PAGE
    i32 = dict(dtype=torch.int32, device="cuda")
    cache = pkv.KVCache(k_buffer=k, v_buffer=v, req_to_token=torch.zeros(2, 1, **i32), req_pool_indices=dev([1]), seq_lens=dev([100]),
                        max_len=512, qo_indptr=dev([0, 40]))
    small = [x[:, BASE:].clone() for x in (k, v)]
    want = P.copy_pages(*(x.view(torch.int32).cpu().numpy() for x in small), None, PAGE, [5, 9], [60, 61])
    pkv.copy_pages(cache, PAGE, dev([first + 5, first + 9]), dev([first + 60, first + 61]))
    for x, w in zip((k, v), want):
        assert np.array_equal(x[:, BASE:].contiguous().view(torch.int32).cpu().numpy(), w)
    table = torch.full((2, 40), -1, **i32)
    table[0, :7] = dev(first + np.arange(20, 27))
    shares = torch.zeros(k.shape[1] // PAGE, **i32)
    end = torch.zeros(1, **i32)
    pkv.fork_requests(cache, table, PAGE, dev([0]), shares, dev([first + 63]), dev([0]), end, token_table=False)
    t = host(table)
    assert (t[1, :6] == t[0, :6]).all() and t[1, 6] == first + 63 and int(shares.sum()) == 6 and int(end) == 1
    for x in (k, v):
        assert torch.equal(x[:, (first + 63) * PAGE:][:, :4], x[:, (first + 26) * PAGE:][:, :4])
        assert (x[:, :2 * TAIL * PAGE] == 0).all()
    for max_q, q_len in ((40, 40), (300, 300)):
        n = 400
        table[0, :32] = dev(first + np.arange(32))
        c = pkv.KVCache(k_buffer=k, v_buffer=v, req_to_token=cache.req_to_token, req_pool_indices=dev([0]), seq_lens=dev([n]), max_len=512,
                        qo_indptr=dev([0, q_len]))
        q = torch.randn(q_len, 2 * kv, d, device="cuda").to(dtype)
        near = Case(pkv.KVCache(k_buffer=k[:, BASE:].contiguous(), v_buffer=v[:, BASE:].contiguous(), req_to_token=cache.req_to_token,
                                req_pool_indices=dev([0]), seq_lens=dev([n]), max_len=512, qo_indptr=dev([0, q_len])),
                    dev([np.arange(32)]), PAGE, q, 1, max_q)
        o = pkv.paged_chunk(c, 1, table, PAGE, q, max_q, workspace=pkv.chunk_workspace(c, q_len, 2 * kv, max_q))
        assert torch.equal(o, near.run(workspace=near.workspace()))
        assert torch.isfinite(o).all()
    assert pkv.last_device_error()[0] == _lib.PKV_OK
