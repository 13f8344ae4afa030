"""Attention of new tokens through the page table on the GPU against its fp64
oracle.

Tolerance per output o of a softmax-weighted mean of values v, with A the
largest sum_c |q_c k_c| |scale| of a pair and n positions: a score is a sum of D
products in fp32, off by D 2^-23 A at most, and by 2^-23 A each for its scaling
and its difference to the maximum, so a weight is off by the factor
exp((D + 2) 2^-23 A) at most, and by 2^-21 for the exponential; numerator and
denominator both, so twice; their sums of n positions, and the factors that
rescale them, n 2^-23 each; bf16 rounds each weight of the numerator by half a
step, 2^-8; the output's rounding is half a step, 2^-8 |o| in bf16 and 2^-24 |o|
in fp32:
  |err| <= max|v| (2 (D + 2) 2^-23 A + 2^-20 + 4 n 2^-23 + [bf16] 2^-8) + half a step.
"""
import dataclasses
import math

import numpy as np
import pytest
import torch

import paged_kv_cache_loc_gb300 as pkv
from oracle import pages_oracle as P
from paged_kv_cache_loc_gb300 import _lib, build

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f32": torch.float32}
DTYPES = ["f32", "bf16"]


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
    return t.double().cpu().numpy() if t.is_floating_point() else t.cpu().numpy().astype(np.int64)


def clean():
    status, detail = pkv.last_device_error()
    assert status == _lib.PKV_OK, detail


def error():
    status, detail = pkv.last_device_error()
    assert status == _lib.PKV_ERR_INDEX
    return detail


@dataclasses.dataclass
class Case:
    cache: object
    table: object
    ps: int
    q: object
    layer: int
    max_q: int

    def run(self, causal=True, **kw):
        return pkv.paged_chunk(self.cache, self.layer, self.table, self.ps, self.q, kw.pop("max_q", self.max_q), causal=causal, **kw)

    def workspace(self):
        return pkv.chunk_workspace(self.cache, self.q.shape[0], self.q.shape[1], self.max_q)

    @property
    def scale(self):
        return 1 / math.sqrt(self.q.shape[2])


def case(q_lens, lens, dtype="f32", kv=2, G=4, d=128, ps=16, layers=1, layer=0, spare_rows=0, spare_pages=3, seed=0, sharp=1.0,
         fill=float("nan")):
    """Entries of random pages in random order.  Every slot that no entry's
    context holds is `fill`."""
    rng = np.random.default_rng(seed + len(q_lens) + ps)
    lens, q_lens = np.asarray(lens), np.asarray(q_lens)
    b, dt = len(lens), DT[dtype]
    held = -(-lens // ps)
    n_pages = int(held.sum()) + spare_pages
    perm, rows = rng.permutation(n_pages), rng.permutation(b + 2)
    table = np.full((b + 2, int(held.max(initial=0)) + 2), -1)
    at = 0
    kept = np.zeros(n_pages * ps, bool)
    for i in range(b):
        table[rows[i], :held[i]] = perm[at:at + held[i]]
        at += held[i]
        pos = np.arange(lens[i])
        kept[table[rows[i], pos // ps] * ps + pos % ps] = True
    g = torch.Generator("cuda").manual_seed(seed + 1)
    k, v = (torch.randn(layers, n_pages * ps, kv, d, generator=g, device="cuda").to(dt) for _ in range(2))
    k[:, ~torch.from_numpy(kept).cuda()] = fill
    v[:, ~torch.from_numpy(kept).cuda()] = fill
    n_q = int(q_lens.sum()) + spare_rows
    q = (torch.randn(n_q, kv * G, d, generator=g, device="cuda") * sharp).to(dt)
    cache = pkv.KVCache(k_buffer=k, v_buffer=v, req_to_token=dev(np.zeros((b + 2, 1))), req_pool_indices=dev(rows[:b]), seq_lens=dev(lens),
                        qo_indptr=dev(np.r_[0, np.cumsum(q_lens)]), max_len=int(lens.max(initial=0)))
    return Case(cache, dev(table), ps, q, layer, int(q_lens.max(initial=0)))


def want(c, causal=True, scale=None, o=None):
    """(the oracle's o, the tolerance of each of its values)."""
    x = c.cache
    base = np.zeros(c.q.shape) if o is None else host(o)
    ref, a, largest = P.chunk(host(x.k_buffer[c.layer]), host(x.v_buffer[c.layer]), host(c.table), c.ps, host(x.req_pool_indices),
                              host(x.seq_lens), host(x.qo_indptr), host(c.q), causal, c.scale if scale is None else scale, base)
    d, n, bf16 = c.q.shape[2], x.max_len, c.q.dtype == torch.bfloat16
    rel = 2 * (d + 2) * 2**-23 * a + 2**-20 + 4 * n * 2**-23 + (2**-8 if bf16 else 0)
    return ref, largest * rel + np.abs(ref) * (2**-8 if bf16 else 2**-24) + 1e-37


def check(got, ref, tol):
    got = host(got)
    assert np.isfinite(got).all()
    over = np.abs(got - ref) - tol
    assert over.max(initial=-1) <= 0, (over.max(), np.unravel_index(over.argmax(), over.shape))


RAGGED = ([0, 1, 5, 64, 65, 130], [7, 1, 90, 64, 500, 131])


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("G,ps", [(1, 16), (2, 1), (4, 24), (8, 128), (4, 8), (1, 3), (4, 256)])
def test_ragged(dtype, causal, d, G, ps):
    c = case(*RAGGED, dtype=dtype, G=G, d=d, ps=ps, kv=2)
    ref, tol = want(c, causal)
    check(c.run(causal), ref, tol)
    check(c.run(causal, workspace=c.workspace()), ref, tol)
    clean()


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("q_lens,lens", [([5, 40, 3, 300, 1], [2, 0, 1, 100, 0]), ([1], [0]), ([129], [128]), ([700, 2], [1, 129])])
def test_contexts_shorter_than_the_rows(dtype, causal, q_lens, lens):
    """Causal rows that see nothing give 0; not causal, lengths need not agree."""
    c = case(q_lens, lens, dtype=dtype)
    ref, tol = want(c, causal)
    o = torch.full_like(c.q, float("nan"))
    check(c.run(causal, o=o), ref, tol)
    o.fill_(float("nan"))
    check(c.run(causal, o=o, workspace=c.workspace()), ref, tol)
    clean()
    if causal:
        first = [i for b in range(len(lens)) for i in range(sum(q_lens[:b]), sum(q_lens[:b]) + max(0, q_lens[b] - lens[b]))]
        assert (o[first] == 0).all()


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("q_len", [1, 2, 8, 31, 100])
@pytest.mark.parametrize("G", [1, 8])
@pytest.mark.parametrize("causal", [True, False])
def test_long_contexts_are_split(dtype, q_len, G, causal):
    c = case([q_len, 1], [4500, 777], dtype=dtype, G=G, kv=1, ps=32)
    ws = c.workspace()
    assert ws.max_splits > 4
    ref, tol = want(c, causal)
    check(c.run(causal, workspace=ws), ref, tol)
    check(c.run(causal), ref, tol)
    few = pkv.Workspace(q_len + 1, G, 128, 3)
    check(c.run(causal, workspace=few), ref, tol)
    clean()


@pytest.mark.parametrize("dtype", DTYPES)
def test_sharp_softmax(dtype):
    """Scores over a wide range: the running maximum is raised many times, and
    most weights vanish."""
    c = case([70, 300], [1500, 300], dtype=dtype, sharp=12.0)
    ref, tol = want(c)
    check(c.run(), ref, tol)
    check(c.run(workspace=c.workspace()), ref, tol)
    clean()


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("scale", [0.0, -0.1, 1.5])
def test_scales(dtype, scale):
    c = case([70, 3], [200, 3000], dtype=dtype, d=64)
    ref, tol = want(c, scale=scale)
    check(c.run(sm_scale=scale), ref, tol)
    check(c.run(sm_scale=scale, workspace=c.workspace()), ref, tol)
    clean()


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("G,q_lens,lens", [(4, [150], [400]), (1, [300], [310]), (8, [5], [2000]), (1, [3, 1], [1000, 129])])
def test_what_is_not_seen_has_no_part(dtype, bad, causal, G, q_lens, lens):
    """Values that are not finite behind the context, in pages of nobody, and
    (causal) at positions of later tokens, row by row."""
    c = case(q_lens, lens, dtype=dtype, G=G, kv=2, fill=bad, seed=5)
    ref, tol = want(c, causal)
    check(c.run(causal, workspace=c.workspace()), ref, tol)
    if causal:
        # position n - 3 of entry 0, in K and in one channel of V: rows before it are as they were
        row, n, q = int(c.cache.req_pool_indices[0]), lens[0], q_lens[0]
        j = n - 3
        slot = int(c.table[row, j // c.ps]) * c.ps + j % c.ps
        c.cache.v_buffer[0, slot, 1, 7] = bad
        got = host(c.run(causal, workspace=c.workspace()))
        sees = np.zeros(c.q.shape[0], bool)
        sees[max(0, q - 3):q] = True
        assert (np.abs(got - ref) <= tol)[~sees].all()
        assert not np.isfinite(got[sees][:, G:, 7]).any()
        if math.isinf(bad):
            assert (got[sees][:, G:, 7] == bad).all()
        keep = np.ones_like(got, bool)
        keep[sees, G:, 7] = False
        assert (np.abs(got - ref) <= tol)[keep].all()
        c.cache.v_buffer[0, slot, 1, 7] = 0
        c.cache.k_buffer[0, slot, 0, 3] = float("nan")
        got = host(c.run(causal, workspace=c.workspace()))
        ref, tol = want(dataclasses.replace(c, cache=dataclasses.replace(c.cache, k_buffer=torch.nan_to_num(c.cache.k_buffer))), causal)
        assert np.isnan(got[sees][:, :G]).all()
        assert (np.abs(got - ref) <= tol)[~sees].all()
    clean()


@pytest.mark.parametrize("dtype", DTYPES)
def test_rows_of_no_entry_stay(dtype):
    """Rows behind the last entry, and between entries that do not touch."""
    c = case([10, 20, 200], [30, 20, 300], dtype=dtype, spare_rows=50)
    o = torch.full_like(c.q, 3.25)
    ref, tol = want(c, o=o)
    check(c.run(o=o), ref, tol)
    assert (o[230:] == 3.25).all()
    o.fill_(3.25)
    check(c.run(o=o, workspace=pkv.Workspace(280, 8, 128, 8)), ref, tol)
    assert (o[230:] == 3.25).all()
    clean()


@pytest.mark.parametrize("dtype", DTYPES)
def test_other_layers_and_many_heads(dtype):
    for kv in (3, 16):
        c = case([33, 2], [100, 700], dtype=dtype, kv=kv, G=2, d=64, layers=3, layer=2, ps=8)
        ref, tol = want(c)
        check(c.run(), ref, tol)
    clean()


@pytest.mark.parametrize("dtype", DTYPES)
def test_many_entries(dtype):
    rng = np.random.default_rng(3)
    c = case(rng.integers(0, 4, 300), rng.integers(0, 90, 300), dtype=dtype, d=64, kv=1, G=2)
    ref, tol = want(c)
    check(c.run(workspace=c.workspace()), ref, tol)
    empty = dataclasses.replace(c, q=c.q[:0], cache=dataclasses.replace(c.cache, req_pool_indices=dev([]), seq_lens=dev([]), qo_indptr=dev([0])))
    assert empty.run().shape == (0, 2, 64)
    clean()


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("causal", [True, False])
def test_many_entries_of_many_rows(dtype, causal):
    """More entries than a warp has lanes, some without rows, in an order of
    lengths with equal ones, and one of the later ones with an error."""
    rng = np.random.default_rng(4)
    q_lens = rng.integers(0, 160, 70) * (rng.integers(0, 5, 70) > 0)
    q_lens[50] = 159
    c = case(q_lens, rng.integers(0, 6, 70) * 61, dtype=dtype, d=64, kv=1, G=2)
    o = torch.full_like(c.q, 2.5)
    ref, tol = want(c, causal, o=o)
    check(c.run(causal, o=o), ref, tol)
    clean()
    c.cache.seq_lens[50] = -7
    o.fill_(2.5)
    c.run(causal, o=o)
    assert error() == -7
    got, lo = host(o), int(q_lens[:50].sum())
    assert (got[lo:lo + 159] == 2.5).all()
    assert (np.abs(got - ref) <= tol)[:lo].all() and (np.abs(got - ref) <= tol)[lo + 159:].all()


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("what,value", [("row", 99), ("row", -1), ("len", -1), ("len", 10**6), ("rows", 10**6), ("rows", -5), ("back", 0)])
def test_bad_entry_is_left_out(dtype, what, value):
    c = case([10, 20, 30], [50, 60, 70], dtype=dtype)
    o = torch.full_like(c.q, 2.5)
    ref, tol = want(c, o=o)
    x = c.cache
    lo, hi = 10, 30
    if what == "row":
        x.req_pool_indices[1] = value
        detail = value
    elif what == "len":
        x.seq_lens[1] = value
        detail = value
    elif what == "rows":                          # the first and second, or second and third, entry's border
        x.qo_indptr[2 if value > 0 else 1] = value
        lo, hi, detail = (10, 60, value) if value > 0 else (0, 30, value)
    else:                                         # more rows than max_q_len
        detail = 30
    kw = dict(max_q=25) if what == "back" else {}
    if what == "back":
        lo, hi = 30, 60
    for ws in (None, pkv.Workspace(60, 8, 128, 8)):
        o.fill_(2.5)
        c.run(o=o, workspace=ws, **kw)
        assert error() == detail
        got = host(o)
        assert (got[lo:hi] == 2.5).all()
        assert (np.abs(got - ref) <= tol)[:lo].all() and (np.abs(got - ref) <= tol)[hi:].all()


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("page", [-1, 10**6])
def test_bad_page_is_reported(dtype, page):
    c = case([10, 20], [100, 200], dtype=dtype, fill=0.5)
    ref, tol = want(c)
    c.table[int(c.cache.req_pool_indices[0]), 2] = page
    got = c.run()
    assert error() == page
    check(got[10:], ref[10:], tol[10:])


@pytest.mark.parametrize("dtype", DTYPES)
def test_streams_and_graphs(dtype):
    """A captured call follows its inputs; two calls on two streams with a
    workspace each do not meet."""
    c = case([8, 8], [3000, 2500], dtype=dtype, kv=1)
    ref, tol = want(c)
    ws, ws2, o, o2 = c.workspace(), c.workspace(), torch.zeros_like(c.q), torch.zeros_like(c.q)
    c.run(o=o, workspace=ws)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for _ in range(10):
        c.run(o=o, workspace=ws)
        c.run(o=o2, workspace=ws2, stream=side)
    torch.cuda.synchronize()
    check(o, ref, tol)
    assert torch.equal(o, o2)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        c.run(o=o, workspace=ws)
    c.cache.seq_lens.copy_(dev([2000, 100]))
    c.q.mul_(0.5)
    ref, tol = want(c)
    g.replay()
    check(o, ref, tol)
    first = o.clone()
    g.replay()
    assert torch.equal(o, first)
    clean()


@pytest.mark.parametrize("dtype", DTYPES)
def test_few_rows_beside_many(dtype):
    """Single tokens with long contexts in the batch of a prompt's chunk, and a
    prompt of its own length beside an entry without rows."""
    c = case([1, 300, 1, 0, 129], [900, 400, 33, 70, 129], dtype=dtype, kv=1)
    ref, tol = want(c)
    check(c.run(), ref, tol)
    check(c.run(workspace=c.workspace()), ref, tol)
    clean()


@pytest.mark.parametrize("dtype", DTYPES)
def test_contexts_that_two_ctas_share(dtype):
    """Contexts of 4096 positions and more, entries of one to five pairs of
    query tiles, causal and not."""
    c = case([70, 600, 129, 200], [4200, 4500, 300, 129], dtype=dtype, kv=1, G=2, d=64)
    for causal in (True, False):
        ref, tol = want(c, causal)
        check(c.run(causal), ref, tol)
    for ps in (1, 8, 128):
        c = case([300], [4100], dtype=dtype, kv=1, G=2, d=128, ps=ps)
        ref, tol = want(c)
        check(c.run(workspace=c.workspace()), ref, tol)
    clean()


@pytest.mark.parametrize("dtype", DTYPES)
def test_long_contexts_that_no_ctas_share(dtype):
    """One query tile, and an odd number of them in so many entries that empty
    partners would not fit beside the others."""
    c = case([100], [4500], dtype=dtype, kv=1, G=2, d=64)
    ref, tol = want(c)
    check(c.run(), ref, tol)
    check(c.run(workspace=c.workspace()), ref, tol)
    c = case([300] + [257] * 39, [4100] + [300] * 39, dtype=dtype, kv=1, G=2, d=64)
    ref, tol = want(c)
    check(c.run(), ref, tol)
    clean()


@pytest.mark.parametrize("dtype", DTYPES)
def test_workspace_that_is_none(dtype):
    c = case([8], [3000], dtype=dtype)
    ws = c.workspace()
    ws.desc.magic = 0
    with pytest.raises(pkv.PkvError) as e:
        c.run(workspace=ws)
    assert e.value.status == _lib.PKV_ERR_WORKSPACE
    clean()


@pytest.mark.parametrize("dtype", DTYPES)
def test_pinned_host_memory(dtype):
    c = case([8, 3], [300, 250], dtype=dtype)
    ref, tol = want(c)
    c.q = c.q.cpu().pin_memory()
    o = torch.zeros(c.q.shape, dtype=c.q.dtype).pin_memory()
    c.run(o=o)
    clean()
    check(o, ref, tol)


@pytest.mark.parametrize("dtype", DTYPES)
def test_agrees_with_decode_over_pages(dtype):
    if dtype == "f32":
        pytest.skip("decode by page table is bf16 alone")
    c = case([1, 1, 1], [100, 2000, 17], dtype=dtype, kv=8)
    ref, tol = want(c)
    ws = pkv.Workspace(3, 32, 128, 64)
    check(pkv.paged_decode_pages(c.cache, 0, c.table, c.ps, c.q, workspace=ws), ref, tol)
    check(c.run(workspace=ws), ref, tol)


def test_refusals():
    c = case([8, 8], [300, 250])
    x = c.cache
    with pytest.raises(ValueError, match="qo_indptr"):
        dataclasses.replace(c, cache=dataclasses.replace(x, qo_indptr=None)).run()
    with pytest.raises(ValueError, match="qo_indptr must have 3"):
        dataclasses.replace(c, cache=dataclasses.replace(x, qo_indptr=dev([0, 8]))).run()
    with pytest.raises(ValueError, match="q must be"):
        dataclasses.replace(c, q=c.q[:, :, :64].contiguous()).run()
    with pytest.raises(TypeError, match="q must be"):
        dataclasses.replace(c, q=c.q.half()).run()
    with pytest.raises(ValueError, match="contiguous"):
        dataclasses.replace(c, q=c.q[::2]).run()
    with pytest.raises(ValueError, match="o must be"):
        c.run(o=c.q[:3])
    with pytest.raises(ValueError, match="req_to_page"):
        dataclasses.replace(c, table=c.table[0]).run()
    for change in (dict(q=c.q[:, :3].contiguous()), dict(ps=7), dict(ps=0), dict(layer=1), dict(layer=-1),
                   dict(cache=dataclasses.replace(x, max_len=10**6)), dict(q=c.q[:, :6].contiguous()), dict(max_q=65535 * 64), dict(max_q=-1)):
        with pytest.raises(pkv.PkvError):
            dataclasses.replace(c, **change).run()
    for scale in (float("nan"), float("inf")):
        with pytest.raises(pkv.PkvError):
            c.run(sm_scale=scale)
    with pytest.raises(pkv.PkvError):
        c.run(o=c.q)
    with pytest.raises(ValueError, match="refuses"):
        pkv.chunk_workspace(x, 16, 6, 8)
    clean()


def test_a_run_of_the_page_operators():
    """A prompt in two chunks, three samples forked from it that each verify a
    draft, the drafts cut back, one sample ended, the pool compacted: the
    attention of every sample is what its own tokens say, and moving the pages
    changes no bit of it."""
    ps, layers, kv, G, d, n_pages = 16, 2, 2, 4, 128, 64
    gen = torch.Generator("cuda").manual_seed(1)
    rng = np.random.default_rng(1)

    def rnd(*shape):
        return torch.randn(*shape, generator=gen, device="cuda").to(torch.bfloat16)

    def zeros(n):
        return torch.zeros(n, dtype=torch.int32, device="cuda")

    pool = [torch.full((layers, n_pages * ps, kv, d), float("nan"), dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    table, tokens = dev(np.full((5, 16), -1)), dev(np.full((5, 256), -1))
    free, shares, places = dev(rng.permutation(n_pages)), zeros(n_pages), [zeros(1), zeros(1)]
    history = {0: [[], []]}                                    # row -> its K and V rows, per layer

    def cache(rows, lens, n_new=0, q_lens=None):
        c = pkv.KVCache(k_buffer=pool[0], v_buffer=pool[1], req_to_token=tokens, req_pool_indices=dev(rows), seq_lens=dev(lens),
                        out_cache_loc=zeros(n_new) if n_new else None, max_len=max(lens), qo_indptr=zeros(len(rows) + 1))
        if q_lens is not None:
            pkv.build_tables(c, table, ps, free, places[0], places[1], q_lens=dev(q_lens))
            places.reverse()
        return c

    def add(rows, lens, q_lens):
        """New tokens of the rows, written and attended to; checked in 64 bits."""
        n = sum(q_lens)
        c = cache(rows, lens, n, q_lens)
        q = rnd(n, kv * G, d)
        for layer in range(layers):
            k, v = rnd(n, kv, d), rnd(n, kv, d)
            pkv.kv_write(c, layer, k, v)
            at = 0
            for r, m in zip(rows, q_lens):
                for x, new in zip(history[r], (k, v)):
                    x.append((layer, new[at:at + m]))
                at += m
            look(c, rows, q, layer, max(q_lens))
        return c, q

    def look(c, rows, q, layer, max_q):
        ws = pkv.chunk_workspace(c, q.shape[0], kv * G, max_q)
        o = pkv.paged_chunk(c, layer, table, ps, q, max_q, workspace=ws)
        clean()
        at, indptr = 0, host(c.qo_indptr)
        for i, r in enumerate(rows):
            k, v = (torch.cat([x for l, x in history[r][u] if l == layer]) for u in range(2))
            m = int(indptr[i + 1] - indptr[i])
            one = dataclasses.replace(c, k_buffer=k[None], v_buffer=v[None], req_pool_indices=dev([0]), seq_lens=dev([len(k)]),
                                      qo_indptr=dev([0, m]), max_len=len(k))
            alone = Case(one, dev([np.arange(len(k))]), 1, q[at:at + m], 0, m)
            ref, tol = want(alone)
            check(o[at:at + m], ref, tol)
            at += m
        return o

    add([0], [70], [70])
    add([0], [101], [31])
    start = int(places[0])
    # three samples of the prompt; the third takes over 96 positions, whole pages alone
    history.update({r: [list(x) for x in history[0]] for r in (1, 2)})
    third = [[(l, x[:max(0, 96 - before)]) for (l, x), before in zip(history[0][u], [0, 0, 70, 70])] for u in range(2)]
    history[3] = third
    pkv.fork_requests(cache([1, 2, 3], [101, 101, 96]), table, ps, dev([0, 0, 0]), shares, free, places[0], places[1])
    places.reverse()
    clean()
    assert int(places[0]) == start + 2 and host(shares).sum() == 3 * 6
    c, q = add([0, 1, 2, 3], [109, 104, 117, 97], [8, 3, 16, 1])
    # of the drafts 2, 1, 5 and 1 tokens stay
    keep = [103, 102, 106, 97]
    pkv.release_pages(cache([0, 1, 2, 3], [109, 104, 117, 97]), table, ps, shares, free, places[0], places[1], dev(keep))
    places.reverse()
    clean()
    for r, n in zip(range(4), keep):
        for u in range(2):
            per = {l: torch.cat([x for k, x in history[r][u] if k == l])[:n] for l in range(layers)}
            history[r][u] = list(per.items())
    c, q = add([0, 1, 2, 3], [n + 2 for n in keep], [2] * 4)
    before = [look(c, [0, 1, 2, 3], q, layer, 2) for layer in range(layers)]
    # row 1 ends, and the used pages move to the front
    pkv.release_pages(cache([1], [104]), table, ps, shares, free, places[0], places[1])
    places.reverse()
    used = n_pages - (n_pages - int(places[0]))
    remap = pkv.compact_pages(cache([0], [1]), table, ps, shares, free, places[0], workspace=pkv.compact_workspace(n_pages))
    clean()
    t = host(table)
    assert (t[1] == -1).all() and t.max() < used == len({p for p in t.flatten() if p >= 0})
    assert (host(remap) < n_pages).all()
    three = [0, 2, 3]
    c3 = cache(three, [keep[r] + 2 for r in three])
    c3.qo_indptr = dev([0, 2, 4, 6])
    q3 = torch.cat([q[2 * r:2 * r + 2] for r in three])
    for layer in range(layers):
        o = look(c3, three, q3, layer, 2)
        for i, r in enumerate(three):
            # the same pieces of each context, so the same sums
            alone = [cache([r], [keep[r] + 2]) for _ in range(1)][0]
            alone.qo_indptr = dev([0, 2])
            a = pkv.paged_chunk(alone, layer, table, ps, q[2 * r:2 * r + 2].contiguous(), 2)
            assert torch.equal(a, pkv.paged_chunk(alone, layer, table, ps, q[2 * r:2 * r + 2].contiguous(), 2))
            assert torch.allclose(o[2 * i:2 * i + 2].float(), before[layer][2 * r:2 * r + 2].float(), atol=0.05)
