"""Cases of the sparse decode path: the step's tables, the pages' key bounds,
the selection of pages, the attention over them, and the step that runs the
last three after the cache write.

Every operator has two forms on the same state: `own` calls
paged_kv_cache_loc_gb300's entry points, the other computes the definition with
elementary torch operations (32-bit attention and bounds, 64-bit scores, since
pages next to the selection's border are told apart by their scores' last
bits).

Operators (all over a pool of pages of `page` consecutive slots):
  tables  per entry, pages for its new tokens from a free list, in entry order;
          prefix sums of the lengths, positions and slots of the new tokens
  bounds  per page and kv head, the channelwise minimum and maximum of its keys
  select  per entry and kv head, the top_k pages by the largest product that
          any of the group's query heads can reach within the page's bounds
  attend  decode attention over the selected pages of each kv head
  step    cache write, bounds, select and attend
"""
import math

import numpy as np
import torch

own = False

DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def _case(name, op, **kw):
    c = dict(name=name, op=op, dtype="bf16", heads=32, kv_heads=8, head_dim=128, page=16, batch=1,
             ctx_lo=1, ctx_hi=1, new_lo=1, new_hi=1, top_k=64, first=1, last=2, prompt=False)
    c.update(kw)
    return c


def listed():
    return [
        # every decode step of a serving loop: 64 running requests take one slot each
        _case("tables_decode_b64", "tables", batch=64, ctx_lo=511, ctx_hi=4095),
        # a large admission: 256 prompts with cached prefixes, 278K new tokens
        _case("tables_prefill_b256", "tables", batch=256, ctx_lo=0, ctx_hi=4096, new_lo=128, new_hi=2048),
        # the bounds after a decode step's write, one new key per request
        _case("bounds_decode_b32", "bounds", batch=32, ctx_lo=511, ctx_hi=4095),
        # the bounds after the write of a ragged prefill batch of 16 prompts
        _case("bounds_prefill_b16", "bounds", batch=16, ctx_lo=0, ctx_hi=4096, new_lo=128, new_hi=2048),
        # batched decode at the contexts of the dense benchmark
        _case("select_b32_4k", "select", batch=32, ctx_lo=512, ctx_hi=4096),
        # long-context serving: few requests, tens of thousands of positions each
        _case("select_b16_128k", "select", batch=16, ctx_lo=32768, ctx_hi=131072, page=32, top_k=128),
        # one interactive request at 32K positions: latency
        _case("attend_b1_32k", "attend", ctx_lo=32768, ctx_hi=32768, top_k=128),
        # a full serving batch: 2048 positions of each kv head of each request
        _case("attend_b64_16k", "attend", batch=64, ctx_lo=4096, ctx_hi=16384, top_k=128),
        # fp32 cache of a small model, odd page size, contexts shorter than the selection among them
        _case("attend_f32_odd_pages", "attend", dtype="f32", heads=8, kv_heads=2, head_dim=64, page=24, batch=13,
              ctx_lo=1, ctx_hi=1777, top_k=20),
        # the whole step of one interactive request
        _case("step_b1_32k", "step", ctx_lo=32767, ctx_hi=32767),
        # the whole step of a small batch
        _case("step_b16_4k", "step", batch=16, ctx_lo=1023, ctx_hi=4095),
        # a chunk of one prompt: 256 queries, each an entry that sees the positions up to its own
        _case("step_prompt_256", "step", batch=256, ctx_lo=16000, ctx_hi=16000, prompt=True),
    ]


def draw(rng):
    def log(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    op = rng.choice(["tables", "bounds", "select", "attend", "step"])
    page = rng.choice([1, 8, 16, 16, 24, 32, 64, 128])
    batch = log(1, 64)
    group, kv = rng.choice([1, 2, 4, 8]), rng.choice([1, 2, 3, 4, 8])
    c = _case("", op, dtype=rng.choice(["bf16", "bf16", "bf16", "f32"]), heads=group * kv, kv_heads=kv,
              head_dim=rng.choice([64, 128]), page=page, batch=batch)
    if op in ("tables", "bounds"):
        c["ctx_hi"] = log(1, 8192)
        c["ctx_lo"] = rng.randint(0, c["ctx_hi"])
        if rng.random() < 0.6:
            c["new_hi"] = log(2, 2048)
            c["new_lo"] = rng.randint(0, c["new_hi"])
    else:
        most = min(65536, 524288 // batch, 50000 * page // batch) if op != "step" else min(32768, 65536 // batch)
        c["first"], c["last"] = rng.randint(0, 2), rng.randint(1, 3)
        c["top_k"] = c["first"] + c["last"] + log(4, max(5, min(256, 2048 // page, most // (16 * page))))
        # a selection leaves most pages of the longest entry out; attention also meets lists that hold every page
        least = 4 * c["top_k"] * page if op == "select" else 1
        c["ctx_hi"] = log(least, max(most, least + 1))
        c["ctx_lo"] = rng.randint(1, c["ctx_hi"])
        if op == "step" and rng.random() < 0.25:
            c["prompt"] = True
            c["batch"] = log(2, 256)
            c["ctx_lo"] = c["ctx_hi"] = log(1, min(16384, 1024 * page))
    del c["name"]
    return c


def _spread(lo, hi, n):
    """n whole lengths evenly over [lo, hi]: their sum does not depend on the seed, their order does."""
    return np.array([lo + (hi - lo) * i // max(1, n - 1) for i in range(n)], np.int64) if n > 1 else np.array([hi], np.int64)


def _lengths(case):
    """(positions before the new tokens, new tokens) of each entry, unpermuted."""
    n = case["batch"]
    old = _spread(case["ctx_lo"], case["ctx_hi"], n)
    if case["op"] in ("select", "attend"):
        return old, np.zeros(n, np.int64)
    if case["op"] == "step":
        return (np.full(n, case["ctx_hi"]) if case["prompt"] else old), np.ones(n, np.int64)
    return old, _spread(case["new_lo"], case["new_hi"], n)


def _rand(gen, *shape):
    return torch.randn(*shape, generator=gen, device="cuda", dtype=torch.float32)


def _keys(gen, n_pages, page, kv, d):
    """Keys as a model makes them: a mean per head and channel with a few large
    channels, a part that the tokens of a page have in common, and the rest."""
    mean = _rand(gen, kv, d) * (1 + 3 * (torch.rand(kv, d, generator=gen, device="cuda") < 0.03))
    out = torch.empty(n_pages * page, kv, d, device="cuda", dtype=torch.bfloat16)
    step = max(1, (1 << 26) // (page * kv * d))
    for p0 in range(0, n_pages, step):
        m = min(step, n_pages - p0)
        x = _rand(gen, m, page, kv, d) * 0.8 + _rand(gen, m, 1, kv, d) * 0.6 + mean
        out[p0 * page:(p0 + m) * page] = x.view(m * page, kv, d)
    return out


def prepare(case, seed):
    gen = torch.Generator("cuda")
    gen.manual_seed(seed)
    rs = np.random.RandomState(seed % (1 << 31))
    dt, op, ps, b = DT[case["dtype"]], case["op"], case["page"], case["batch"]
    kv, heads, d = case["kv_heads"], case["heads"], case["head_dim"]
    old, new = _lengths(case)
    if case["prompt"]:   # one request: entry i sees the positions up to its own
        lens = old + 1 + np.arange(b)
        req_len, req_of = np.array([lens[-1]]), np.zeros(b, np.int64)
    else:
        old, new = rs.permutation(old), rs.permutation(new)
        lens = old + new
        req_len, req_of = lens, np.arange(b)
    n_req = len(req_len)
    rows = rs.permutation(n_req + 3)[:n_req]                 # each request's row of the page table
    np_req = -(-req_len // ps)
    np_old = -(-old // ps) if op == "tables" else np_req     # pages that the requests hold before the call
    max_pages = -(-max(1, case["ctx_hi"] + (b if case["prompt"] else int(new.max()))) // ps)
    n_pages = int(old.sum() + new.sum()) // ps + b + (1000 if op == "tables" else 8) if not case["prompt"] else max_pages + 8
    perm = rs.permutation(n_pages)
    table = np.full((n_req + 3, max_pages), -1, np.int32)
    at = 0
    for i in range(n_req):
        table[rows[i], :np_old[i]] = perm[at:at + np_old[i]]
        at += int(np_old[i])

    def dev(a):
        return torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).cuda()

    s = dict(case=case, max_len=int(lens.max()), table=dev(table), rows=dev(rows[req_of]), lens=dev(lens), n_pages=n_pages,
             max_pages=max_pages)
    n_new = int(new.sum())
    if op == "tables":
        s["q_lens"] = dev(new)
        s["free"] = dev(np.r_[rs.randint(0, n_pages, 5), perm[at:]])   # 5 entries taken by earlier calls
        s["free_start"] = dev([5])
        s["free_end"] = torch.zeros(1, dtype=torch.int32, device="cuda")
        s["token_table"] = torch.zeros(n_req + 3, max_pages * ps, dtype=torch.int32, device="cuda")
        s["kv_indptr"], s["qo_indptr"] = (torch.zeros(b + 1, dtype=torch.int32, device="cuda") for _ in range(2))
        s["loc"], s["positions"] = (torch.full((n_new,), -1, dtype=torch.int32, device="cuda") for _ in range(2))
        s["k"] = torch.empty(1, n_pages * ps, 1, 8, dtype=torch.bfloat16, device="cuda")   # the pool's size alone is used
        s["v"] = s["k"]
    else:
        if op == "select":   # the bounds are all that is read of the keys
            center = _rand(gen, n_pages, kv, d) * 0.6 + _rand(gen, kv, d) * (1 + 3 * (torch.rand(kv, d, generator=gen, device="cuda") < 0.03))
            half = 0.8 * (1.2 + 0.4 * torch.rand(n_pages, kv, 2, d, generator=gen, device="cuda"))
            s["bounds"] = torch.stack([center - half[:, :, 0], center + half[:, :, 1]], 2).to(dt)[None].contiguous()
            s["k"] = torch.empty(1, n_pages * ps, kv, d, dtype=dt, device="cuda")
            s["v"] = s["k"]
        else:
            s["k"] = _keys(gen, n_pages, ps, kv, d).to(dt)[None].contiguous()
            s["v"] = (torch.randn(1, n_pages * ps, kv, d, generator=gen, device="cuda", dtype=torch.bfloat16).to(dt)
                      if op != "bounds" else s["k"])
        pos = np.concatenate([np.arange(o, o + n) for o, n in zip(old, new)]) if not case["prompt"] else lens - 1
        row = np.repeat(rows[req_of], new)
        s["loc"] = dev(table[row, pos // ps].astype(np.int64) * ps + pos % ps) if n_new else dev([])
        if op in ("bounds", "step"):   # bounds of what the pages held before: the new keys' rows left out
            held = torch.zeros(n_pages * ps, dtype=torch.bool, device="cuda")
            for i in range(n_req):
                o = int(old[0]) if case["prompt"] else int(old[i])
                p = np.arange(o)
                held[torch.from_numpy(table[rows[i], p // ps].astype(np.int64) * ps + p % ps).cuda()] = True
            kk = s["k"][0].view(n_pages, ps, kv, d)
            hh = held.view(n_pages, ps, 1, 1)
            lo = torch.where(hh, kk, torch.inf).amin(1)
            hi = torch.where(hh, kk, -torch.inf).amax(1)
            s["bounds"] = torch.where(torch.isfinite(torch.stack([lo, hi], 2)), torch.stack([lo, hi], 2), 0).to(dt)[None].contiguous()
        if op == "step":
            loc = s["loc"].long()
            s["k_new"], s["v_new"] = s["k"][0, loc].clone(), s["v"][0, loc].clone()
            s["k"][0, loc], s["v"][0, loc] = 0, 0
        if op != "bounds":   # queries that look for some of the request's pages
            s["q"] = (_rand(gen, b, heads, d) * 0.7 + _rand(gen, b, kv, 1, d).expand(-1, -1, heads // kv, -1).reshape(b, heads, d)).to(dt)
        if op == "attend":   # a selection as select makes it: the last page and others, in ascending order
            score = torch.rand(b, kv, max_pages, generator=gen, device="cuda")
            p = torch.arange(max_pages, device="cuda")
            n = ((s["lens"] + ps - 1) // ps)[:, None, None]
            score = torch.where(p >= n - 1, torch.where(p >= n, -1.0, 2.0), score)
            k = min(case["top_k"], max_pages)
            best = score.topk(k, -1).indices
            s["counts"] = torch.clamp(n.expand(b, kv, 1), max=case["top_k"])[:, :, 0].to(torch.int32).contiguous()
            best = torch.where(best < n, best, 1 << 30).sort(-1).values
            s["sel"] = torch.full((b, kv, case["top_k"]), -1, dtype=torch.int32, device="cuda")
            s["sel"][:, :, :k] = torch.where(best < (1 << 30), best, -1).to(torch.int32)
    s["scale"] = 1.0 / math.sqrt(d)
    if own:
        import paged_kv_cache_loc_gb300 as pkv
        s["cache"] = pkv.KVCache(k_buffer=s["k"], v_buffer=s["v"], req_to_token=s.get("token_table", s["table"]), req_pool_indices=s["rows"],
                                 seq_lens=s["lens"], out_cache_loc=s.get("loc"), max_len=s["max_len"], kv_indptr=s.get("kv_indptr"),
                                 qo_indptr=s.get("qo_indptr"))
        if op != "tables":
            bounds = s.get("bounds")
            s["pages"] = pkv.SparsePages(page_bounds=bounds, req_to_page=s["table"], page_size=ps, top_k=case["top_k"],
                                         n_first=case["first"], n_last=case["last"])
            need = pkv.select_workspace_bytes(b, kv, s["max_len"], ps)
            s["ws"] = pkv.Workspace(b, heads, d, max(1, -(-need // (b * heads * d * 4))))
    return s


# ---------------------------------------------------------------------------
# plain forms
# ---------------------------------------------------------------------------

def _tables(s):
    ps, lens, q = s["case"]["page"], s["lens"].long(), s["q_lens"].long()
    n_new = s["loc"].numel()
    start = lens - q
    p0, p1 = (start + ps - 1) // ps, (lens + ps - 1) // ps       # new pages [p0, p1) of each entry
    need = p1 - p0
    before = torch.cumsum(need, 0) - need
    s["kv_indptr"][1:] = torch.cumsum(lens, 0)
    s["qo_indptr"][1:] = torch.cumsum(q, 0)
    s["free_end"][:] = s["free_start"] + need.sum()
    b = torch.repeat_interleave(torch.arange(len(q), device=q.device), q, output_size=n_new)
    pos = start[b] + torch.arange(n_new, device=q.device) - (torch.cumsum(q, 0) - q)[b]
    pg = pos // ps
    row = s["rows"].long()[b]
    taken = torch.clamp(s["free_start"].long() + before[b] + pg - p0[b], min=0)
    page = torch.where(pg >= p0[b], s["free"].long()[taken.clamp(max=s["free"].numel() - 1)], s["table"].long()[row, pg])
    s["table"][row, pg] = page.to(torch.int32)
    s["loc"][:] = page * ps + pos % ps
    s["positions"][:] = pos
    s["token_table"][row, pos] = s["loc"]


def _bounds(s, keys):
    """Keys [n, kv, d] at slots s["loc"], in ascending order within a page."""
    ps, loc = s["case"]["page"], s["loc"].long()
    page = loc // ps
    kv, d = keys.shape[1:]
    at = page[:, None, None].expand(-1, kv, d)
    old = s["bounds"][0].float()
    fresh = torch.zeros(s["n_pages"], device=loc.device).index_add(0, page, (loc % ps == 0).float()) > 0
    lo = torch.where(fresh[:, None, None], torch.inf, old[:, :, 0]).scatter_reduce(0, at, keys.float(), "amin")
    hi = torch.where(fresh[:, None, None], -torch.inf, old[:, :, 1]).scatter_reduce(0, at, keys.float(), "amax")
    s["bounds"][0] = torch.stack([lo, hi], 2).to(s["bounds"].dtype)


def _select(s):
    c, ps = s["case"], s["case"]["page"]
    b, kv, d, k = c["batch"], c["kv_heads"], c["head_dim"], c["top_k"]
    q = s["q"].double().view(b, kv, -1, d)
    page = s["table"].long()[s["rows"].long()].clamp(min=0)              # [b, max_pages]
    x = s["bounds"][0][page].permute(0, 2, 3, 1, 4).double()              # [b, kv, 2, max_pages, d]
    score = q.clamp(max=0) @ x[:, :, 0].transpose(-1, -2) + q.clamp(min=0) @ x[:, :, 1].transpose(-1, -2)
    score = score.amax(2)                                                 # [b, kv, max_pages]
    p = torch.arange(s["max_pages"], device=q.device)
    n = ((s["lens"].long() + ps - 1) // ps)[:, None, None]
    score = torch.where((p < c["first"]) | (p >= n - c["last"]), torch.inf, score)
    score = torch.where(p < n, score, -torch.inf)
    best = score.sort(stable=True, dim=-1, descending=True).indices[:, :, :k]   # ties to the lowest page
    best = torch.where(best < n, best, 1 << 30).sort(-1).values
    sel = torch.full((b, kv, k), -1, dtype=torch.int32, device=q.device)
    sel[:, :, :best.shape[2]] = torch.where(best < (1 << 30), best, -1).to(torch.int32)
    return sel, n.clamp(max=k)[:, :, 0].expand(b, kv).to(torch.int32)


def _attend(s, sel):
    c, ps = s["case"], s["case"]["page"]
    b, kv, d = c["batch"], c["kv_heads"], c["head_dim"]
    q = s["q"].float().view(b, kv, -1, d)
    pos = (sel.long()[..., None] * ps + torch.arange(ps, device=q.device)).flatten(2)       # [b, kv, t]
    seen = (pos >= 0) & (pos < s["lens"].long()[:, None, None])
    page = s["table"].long()[s["rows"].long()[:, None, None], sel.long().clamp(min=0)]
    slot = (page[..., None] * ps + torch.arange(ps, device=q.device)).flatten(2)
    slot = torch.where(seen, slot, 0)
    h = torch.arange(kv, device=q.device)[:, None]
    w = q @ s["k"][0][slot, h].float().transpose(-1, -2) * s["scale"]
    w = torch.where(seen[:, :, None], w, -torch.inf)
    w = torch.exp(w - w.amax(-1, keepdim=True).clamp(min=-3e38))
    o = w @ torch.where(seen[..., None], s["v"][0][slot, h].float(), 0)
    o = o / w.sum(-1, keepdim=True).clamp(min=1e-37)
    return o.view(b, -1, d).to(s["q"].dtype)


def _step(s):
    loc = s["loc"].long()
    s["k"][0, loc], s["v"][0, loc] = s["k_new"], s["v_new"]
    _bounds(s, s["k_new"])
    sel, counts = _select(s)
    return _attend(s, sel), sel, counts


def run(s):
    op = s["case"]["op"]
    if op == "tables":
        if own:
            import paged_kv_cache_loc_gb300 as pkv
            pkv.build_tables(s["cache"], s["table"], s["case"]["page"], s["free"], s["free_start"], s["free_end"], s["positions"], s["q_lens"])
        else:
            _tables(s)
        return {k: s[k] for k in ("table", "token_table", "kv_indptr", "qo_indptr", "loc", "positions", "free_end")}
    if op == "bounds":
        if own:
            import paged_kv_cache_loc_gb300 as pkv
            pkv.page_bounds(s["cache"], 0, s["pages"])
        else:
            _bounds(s, s["k"][0][s["loc"].long()])
        return {"bounds": s["bounds"]}
    if op == "select":
        if own:
            import paged_kv_cache_loc_gb300 as pkv
            sel, counts = pkv.select_pages(s["cache"], 0, s["pages"], s["q"], workspace=s["ws"])
        else:
            sel, counts = _select(s)
        return {"sel": sel, "counts": counts}
    if op == "attend":
        if own:
            import paged_kv_cache_loc_gb300 as pkv
            return {"o": pkv.paged_decode_selected(s["cache"], 0, s["pages"], s["q"], s["sel"], s["counts"])}
        return {"o": _attend(s, s["sel"])}
    if own:
        import paged_kv_cache_loc_gb300 as pkv
        o, sel, counts = pkv.sparse_decode_step(s["cache"], 0, s["pages"], s["k_new"], s["v_new"], s["q"], workspace=s["ws"])
    else:
        o, sel, counts = _step(s)
    return {"o": o, "sel": sel, "counts": counts, "bounds": s["bounds"], "k": s["k"], "v": s["v"]}


def work(case):
    """Bytes: each input row read once and each output written once."""
    op, ps, b, kv, d = case["op"], case["page"], case["batch"], case["kv_heads"], case["head_dim"]
    eb = 4 if case["dtype"] == "f32" else 2
    old, new = _lengths(case)
    if op == "tables":
        n, pages = int(new.sum()), int((-(-(old + new) // ps) + -old // ps).sum())
        return {"bytes": 12 * b + 8 * (b + 1) + 12 * n + 8 * pages + 8, "flops": 0}
    lens = case["ctx_hi"] + 1 + np.arange(b) if case["prompt"] else old + new
    pages = -(-lens // ps)
    row = kv * d * eb
    table, q = 4 * int(pages.max() if case["prompt"] else pages.sum()), b * case["heads"] * d * eb
    lists = 4 * b * kv * (case["top_k"] + 1)
    touched = len({(i, int(p)) for i, (o, n) in enumerate(zip(old, new)) for p in range(o // ps, -(-(o + n) // ps))}) if op == "bounds" else 0
    if op == "bounds":
        return {"bytes": int(new.sum()) * (4 + row) + touched * 2 * row + int((old % ps > 0).sum()) * 2 * row, "flops": 2 * int(new.sum()) * kv * d}
    scored = pages[pages > case["top_k"]]            # an entry with fewer pages takes them all
    select = (int(scored.max(initial=0)) if case["prompt"] else int(scored.sum())) * 2 * row + table + q + lists
    select_flops = 4 * d * case["heads"] * int(scored.sum())
    seen = np.minimum(np.minimum(pages, case["top_k"]) * ps, lens)
    rows = min(int(seen.sum()), int(lens.max())) if case["prompt"] else int(seen.sum())
    attend = rows * 2 * row + 2 * q + lists + table
    attend_flops = 4 * d * case["heads"] * int(seen.sum())
    if op == "select":
        return {"bytes": select, "flops": select_flops}
    if op == "attend":
        return {"bytes": attend, "flops": attend_flops}
    return {"bytes": b * (4 * row + 4) + b * 2 * row + select + attend, "flops": select_flops + attend_flops + 2 * b * kv * d}


# ---------------------------------------------------------------------------
# the definitions in 64 bits, entry by entry
# ---------------------------------------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    op, ps, g = case["op"], case["page"], case["heads"] // case["kv_heads"]
    if op == "tables":
        return None   # whole numbers alone
    if op in ("bounds", "step"):
        loc = s["loc"].cpu().numpy().astype(np.int64)
        keys = (s["k_new"] if op == "step" else s["k"][0][s["loc"].long()]).double()
        bounds = s["bounds"].double()
        runs = np.flatnonzero(np.r_[True, (loc[1:] != loc[:-1] + 1) | (loc[1:] % ps == 0)]) if len(loc) else np.zeros(0, np.int64)
        for i, j in zip(runs, np.r_[runs[1:], len(loc)]):
            both = torch.stack([keys[i:j].amin(0), keys[i:j].amax(0)], 1)
            if loc[i] % ps:
                was = bounds[0, loc[i] // ps]
                both = torch.stack([torch.minimum(both[:, 0], was[:, 0]), torch.maximum(both[:, 1], was[:, 1])], 1)
            bounds[0, loc[i] // ps] = both
        if op == "bounds":
            return {"bounds": bounds}
        s["k"][0, s["loc"].long()], s["v"][0, s["loc"].long()] = s["k_new"], s["v_new"]
    else:
        bounds = s["bounds"].double() if op == "select" else None
    b, kv, d = case["batch"], case["kv_heads"], case["head_dim"]
    o = torch.zeros(b, case["heads"], d, dtype=torch.float64, device="cuda")
    rows, lens, table = s["rows"].tolist(), s["lens"].tolist(), s["table"].long()
    lists = s["sel"].cpu().numpy() if op == "attend" else np.full((b, kv, case["top_k"]), -1, np.int32)
    counts = np.zeros((b, kv), np.int32)
    for i in range(b):
        n = -(-lens[i] // ps)
        q = s["q"][i].double().view(kv, g, d)
        for h in range(kv):
            if op != "attend":
                pick = np.arange(n)
                if n > case["top_k"]:
                    x = bounds[0, table[rows[i], :n], h]
                    most = torch.maximum(q[h][:, None] * x[None, :, 0], q[h][:, None] * x[None, :, 1]).sum(-1).amax(0).cpu().numpy()
                    forced = (pick < case["first"]) | (pick >= n - case["last"])
                    order = np.lexsort((pick, -most, ~forced))
                    pick = np.sort(order[:case["top_k"]])
                lists[i, h, :len(pick)], counts[i, h] = pick, len(pick)
            if op == "select":
                continue
            pick = torch.from_numpy(lists[i, h][lists[i, h] >= 0].astype(np.int64)).cuda()
            pos = (pick[:, None] * ps + torch.arange(ps, device="cuda")).flatten()
            slot = (table[rows[i], pick][:, None] * ps + torch.arange(ps, device="cuda")).flatten()[pos < lens[i]]
            if len(slot):
                w = torch.softmax((q[h] @ s["k"][0, slot, h].double().T) / math.sqrt(d), -1)
                o[i, h * g:(h + 1) * g] = w @ s["v"][0, slot, h].double()
    if op == "attend":
        return {"o": o}
    lists, counts = torch.from_numpy(lists).cuda(), torch.from_numpy(counts).cuda()
    if op == "select":
        return {"sel": lists, "counts": counts}
    return {"o": o, "sel": lists, "counts": counts, "bounds": bounds, "k": s["k"].double(), "v": s["v"].double()}
