"""Cases of the life of a cache's pages and of the attention of new tokens over
them: copying, forking, releasing and compacting pages, and chunk attention
through the page table.

Every operator has two forms on the same state: `own` calls
paged_kv_cache_loc_gb300's entry points, the other computes the definition with
elementary torch operations (attention in 32 bits).

Operators (a pool of pages of `page` consecutive slots, `layers` layers):
  copy     page dst[i] becomes a copy of page src[i], K, V and key bounds, every layer
  fork     a child row takes over the first n positions of a parent row: full pages
           are shared (`shares` counts the references beyond the first), a partly
           filled last page is copied to a page of the free list
  release  rows give up their pages behind keep positions; those that nobody shares
           any more go back in front of the free list, in ascending order
  compact  the used pages behind the pool's first U (U pages are used) move to the
           free pages among them; tables, counts and free list follow
  chunk    attention of each entry's new tokens (one to thousands) over its context;
           causal, or over all of it (an encoder's states, of another length)
"""
import math

import numpy as np
import torch

own = False

DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def _case(name, op, **kw):
    c = dict(name=name, op=op, dtype="bf16", heads=32, kv_heads=8, head_dim=128, page=16, batch=1, layers=1,
             ctx_lo=1, ctx_hi=1, new_lo=1, new_hi=1, causal=True, pages=0, moves=0, fan=1, bounds=True)
    c.update(kw)
    return c


def listed():
    return [
        # copy-on-write of one page of each of eight requests, a whole model's layers: latency
        _case("copy_b8", "copy", layers=32, pages=24, moves=8),
        # a host allocator's plan: a thousand pages change places
        _case("copy_1k", "copy", layers=16, pages=2100, moves=1024),
        # eight samples of one prompt, a whole model's layers
        _case("fork_8_of_1", "fork", layers=32, batch=8, fan=8, ctx_lo=1003, ctx_hi=1003),
        # a serving batch: 32 prompts, eight samples of each
        _case("fork_256_of_32", "fork", layers=8, batch=256, fan=8, ctx_lo=512, ctx_hi=4096),
        # after every speculative step: the pages of rejected draft tokens
        _case("release_drafts_b64", "release", batch=64, ctx_lo=512, ctx_hi=4096, new_lo=0, new_hi=12),
        # finished requests at once, prefixes shared by groups of eight
        _case("release_b512", "release", batch=512, fan=8, ctx_lo=2048, ctx_hi=32768, new_lo=2048, new_hi=32768),
        # a small pool after a few requests have ended
        _case("compact_small", "compact", layers=4, batch=16, pages=300, moves=17, ctx_hi=256),
        # a pool that is to shrink: a quarter of its pages change places
        _case("compact_2k", "compact", layers=16, batch=64, pages=2048, moves=500, ctx_hi=2048),
        # one interactive request, a draft of eight tokens to verify at 32K positions: latency
        _case("chunk_draft_b1_32k", "chunk", ctx_lo=32768, ctx_hi=32768, new_lo=8, new_hi=8),
        # chunked prefill: four prompts take 2048 more tokens each
        _case("chunk_prefill_b4_16k", "chunk", batch=4, ctx_lo=8192, ctx_hi=16384, new_lo=2048, new_hi=2048),
        # decoder tokens over an encoder's states, every length different, some longer than the states
        _case("chunk_cross_b16", "chunk", batch=16, heads=16, kv_heads=16, head_dim=64, page=32, ctx_lo=100, ctx_hi=1500,
              new_lo=1, new_hi=448, causal=False),
        # fp32 cache of a small model, odd page size
        _case("chunk_f32_odd_pages", "chunk", dtype="f32", heads=8, kv_heads=2, head_dim=64, page=24, batch=13, ctx_lo=101,
              ctx_hi=1777, new_lo=1, new_hi=101),
    ]


def draw(rng):
    def log(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    op = rng.choice(["copy", "fork", "release", "compact", "chunk", "chunk"])
    group, kv = rng.choice([1, 2, 4, 8]), rng.choice([1, 2, 3, 4, 8])
    c = _case("", op, dtype=rng.choice(["bf16", "bf16", "bf16", "f32"]), heads=group * kv, kv_heads=kv,
              head_dim=rng.choice([64, 128]), page=rng.choice([1, 8, 16, 16, 24, 32, 64, 128]), batch=log(1, 64))
    ps = c["page"]
    row = kv * c["head_dim"] * (4 if c["dtype"] == "f32" else 2)
    if op in ("copy", "compact"):
        c["layers"] = log(1, 32)
        c["bounds"] = rng.random() < 0.5
        most = max(8, min(60000, (1 << 30) // (c["layers"] * 2 * (ps + 1) * row)))
        c["pages"] = log(8, most)
        c["moves"] = log(1, max(2, c["pages"] // (4 if op == "compact" else 2)))
        c["ctx_hi"] = log(1, 4096)
    elif op == "fork":
        c["layers"] = log(1, 32)
        c["fan"] = rng.randint(1, min(8, c["batch"]))
        c["ctx_hi"] = log(1, max(2, min(8192, (1 << 29) // (c["layers"] * 2 * row * c["batch"]))))
        c["ctx_lo"] = rng.randint(0, c["ctx_hi"])
        c["bounds"] = rng.random() < 0.5
    elif op == "release":
        c["batch"] = log(1, 512)
        c["fan"] = rng.randint(1, min(8, c["batch"]))
        c["ctx_hi"] = log(1, 16384)
        c["ctx_lo"] = rng.randint(0, c["ctx_hi"])
        c["new_hi"] = log(1, c["ctx_hi"] + 1)
        c["new_lo"] = rng.randint(0, min(c["new_hi"], c["ctx_lo"]))
    else:
        c["causal"] = rng.random() < 0.75
        budget = (1 << (31 if c["dtype"] == "bf16" else 28)) // (c["heads"] * c["batch"])   # query-key pairs
        c["new_hi"] = log(1, min(2048, math.isqrt(budget)))
        c["new_lo"] = rng.randint(0, c["new_hi"])
        c["ctx_hi"] = log(1, max(2, min(65536, (1 << 20) // c["batch"], budget // c["new_hi"])))
        c["ctx_lo"] = rng.randint(0 if not c["causal"] else 1, c["ctx_hi"])
    del c["name"]
    return c


def _spread(lo, hi, n):
    """n whole lengths evenly over [lo, hi]: their sum does not depend on the seed, their order does."""
    return np.array([lo + (hi - lo) * i // max(1, n - 1) for i in range(n)], np.int64) if n > 1 else np.array([hi], np.int64)


def _lengths(case):
    """(context lengths, new, forked-off or given-up tokens) of each entry, unpermuted."""
    b, fan = case["batch"], case["fan"]
    if case["op"] == "fork":   # the entries of a parent take over the same context
        return np.repeat(_spread(case["ctx_lo"], case["ctx_hi"], -(-b // fan)), fan)[:b], np.zeros(b, np.int64)
    ctx, new = _spread(case["ctx_lo"], case["ctx_hi"], b), _spread(case["new_lo"], case["new_hi"], b)
    if case["op"] == "release":
        new = np.minimum(new, ctx)
    if case["op"] == "chunk" and case["causal"]:
        ctx = np.maximum(ctx, new)     # the new tokens are part of their context
    return ctx, new


def _dev(a):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).cuda()


def _values(gen, *shape, dt):
    """Rows as a model makes them: a few channels larger than the others."""
    out = torch.empty(*shape, device="cuda", dtype=dt)
    scale = 0.8 + 2 * (torch.rand(shape[-2:], generator=gen, device="cuda") < 0.03)
    for part in out.view(-1, *shape[-2:]).split(1 << 18):
        part.copy_(torch.randn(part.shape, generator=gen, device="cuda") * scale)
    return out


def prepare(case, seed):
    gen = torch.Generator("cuda")
    gen.manual_seed(seed)
    rs = np.random.RandomState(seed % (1 << 31))
    dt, op, ps, b = DT[case["dtype"]], case["op"], case["page"], case["batch"]
    kv, heads, d, layers = case["kv_heads"], case["heads"], case["head_dim"], case["layers"]
    s = dict(case=case)
    ctx, new = _lengths(case)
    if op == "copy":
        n_pages = case["pages"]
        perm = rs.permutation(n_pages)
        s["src"], s["dst"] = _dev(perm[:case["moves"]]), _dev(perm[case["moves"]:2 * case["moves"]])
    elif op == "fork":
        n_par = -(-b // case["fan"])
        order = rs.permutation(b)
        par_len = ctx[::case["fan"]]
        rows = rs.permutation(n_par + b + 3)
        held = -(-par_len // ps)
        need = int((ctx % ps > 0).sum())
        n_pages, max_pages = int(held.sum()) + need + 8, int(held.max(initial=0)) + 2
        perm = rs.permutation(n_pages)
        table = np.full((n_par + b + 3, max_pages), -1)
        at = 0
        for i in range(n_par):
            table[rows[i], :held[i]] = perm[at:at + held[i]]
            at += int(held[i])
        s["parents"], s["rows"] = _dev(rows[:n_par][order // case["fan"]]), _dev(rows[n_par:n_par + b])
        s["lens"] = _dev(ctx[order])
        s["shares0"] = _dev(np.bincount(perm[:at // 8], minlength=n_pages))       # some pages are shared already
        s["free"], s["free_start"] = _dev(np.r_[rs.randint(0, n_pages, 5), perm[at:]]), _dev([5])
        s["part"] = (ctx[order] % ps).tolist()
        s["table"] = _dev(table)
        s["max_len"] = int(ctx.max(initial=0))
    elif op == "release":
        order = rs.permutation(b)
        ctx, new = ctx[order], new[order]
        fan = case["fan"]
        held = -(-ctx // ps)
        rows = rs.permutation(b + 3)[:b]
        max_pages = int(held.max(initial=0)) + 1
        n_pages = int(held.sum()) + 64
        perm = rs.permutation(n_pages)
        table = np.full((b + 3, max_pages), -1)
        count = np.zeros(n_pages, np.int64)
        at = 0
        for i in range(b):            # a group's first half of the first member's pages is common
            lead = i - i % fan
            common = min(int(held[i]), int(held[lead]) // 2) if i != lead else 0
            table[rows[i], :common] = table[rows[lead], :common]
            m = int(held[i]) - common
            table[rows[i], common:held[i]] = perm[at:at + m]
            at += m
        np.add.at(count, table[table >= 0], 1)
        s["shares0"] = _dev(np.maximum(count - 1, 0))
        s["rows"], s["lens"], s["keep"], s["table0"] = _dev(rows), _dev(ctx), _dev(ctx - new), _dev(table)
        s["table"] = s["table0"].clone()
        # the pages that are held have been taken from the list's front
        s["free"], s["free_start"] = _dev(np.r_[np.full(at, -1), perm[at:]]), _dev([at])
        s["max_len"] = int(ctx.max(initial=0))
    elif op == "compact":
        n_pages, moves = case["pages"], case["moves"]
        used = n_pages // 2 + moves // 2                       # of them `moves` stand behind the first `used`
        low, high = rs.permutation(used), used + rs.permutation(n_pages - used)
        pages = rs.permutation(np.r_[low[moves:], high[:moves]])
        free = rs.permutation(np.r_[low[:moves], high[moves:]])
        rows_n = b + 3
        width = max(1, min(-(-case["ctx_hi"] // ps), -(-used // b)))
        table = np.full((rows_n, width + 1), -1)
        count = np.zeros(n_pages, np.int64)
        for i in range(b):
            take = pages[i * width:(i + 1) * width]
            table[i, :len(take)] = take
            if i % 3 == 2:                                     # a fork shares its first pages with the row before
                table[i, :min(len(take), width // 2)] = table[i - 1, :min(len(take), width // 2)]
        np.add.at(count, table[table >= 0], 1)
        s["table"], s["shares0"] = _dev(table), _dev(np.maximum(count - 1, 0))
        s["tokens"] = _dev(np.where(table[:, :, None] >= 0, table[:, :, None] * ps + np.arange(ps), -1).reshape(rows_n, -1))
        s["free"], s["free_start"] = _dev(np.r_[rs.randint(0, n_pages, 5), free]), _dev([5])
        s["remap"], s["free_out"] = torch.zeros(n_pages, dtype=torch.int32, device="cuda"), s["free"].clone()
        s["rows"], s["lens"], s["max_len"] = _dev(np.arange(b)), _dev(np.full(b, width * ps)), width * ps
    else:
        order = rs.permutation(b)
        ctx, new = ctx[order], new[rs.permutation(b)] if not case["causal"] else new[order]
        held = -(-ctx // ps)
        rows = rs.permutation(b + 3)[:b]
        n_pages, max_pages = int(held.sum()) + 8, int(held.max(initial=0)) + 1
        perm = rs.permutation(n_pages)
        table = np.full((b + 3, max_pages), -1)
        at = 0
        for i in range(b):
            table[rows[i], :held[i]] = perm[at:at + held[i]]
            at += int(held[i])
        s["table"], s["rows"], s["lens"] = _dev(table), _dev(rows), _dev(ctx)
        s["qo_indptr"] = _dev(np.r_[0, np.cumsum(new)])
        s["ctx"], s["new"], s["max_len"], s["max_q"] = ctx.tolist(), new.tolist(), int(ctx.max()), int(new.max())
        s["q"] = _values(gen, int(new.sum()), heads, d, dt=dt)
    s["n_pages"] = n_pages
    small = op == "release"          # the pool's size alone is used
    s["k"], s["v"] = ((torch.empty(1, n_pages * ps, 1, 8, dtype=torch.bfloat16, device="cuda"),) * 2 if small else
                      [_values(gen, layers, n_pages * ps, kv, d, dt=dt) for _ in range(2)])
    if op in ("copy", "fork", "compact"):
        s["bounds"] = _values(gen, layers, n_pages, kv, 2, d, dt=dt) if case["bounds"] else None
    if op in ("fork", "release", "compact"):
        s["shares"] = s["shares0"].clone()
        s["free_end"] = torch.zeros(1, dtype=torch.int32, device="cuda")
    if op == "fork":
        s["tokens"] = torch.full((s["table"].shape[0], s["table"].shape[1] * ps), -1, dtype=torch.int32, device="cuda")
    if own:
        import paged_kv_cache_loc_gb300 as pkv
        none = _dev([])
        s["cache"] = pkv.KVCache(k_buffer=s["k"], v_buffer=s["v"], req_to_token=s.get("tokens", s.get("table", none)),
                                 req_pool_indices=s.get("rows", none), seq_lens=s.get("lens"), max_len=s.get("max_len", 0),
                                 qo_indptr=s.get("qo_indptr"))
        if op == "compact":
            s["ws"] = pkv.compact_workspace(n_pages)
        if op == "chunk":
            s["ws"] = pkv.chunk_workspace(s["cache"], s["q"].shape[0], heads, s["max_q"])
    return s


# ---------------------------------------------------------------------------
# plain forms
# ---------------------------------------------------------------------------

def _by_page(x, s):
    return x.view(x.shape[0], s["n_pages"], -1)


def _copy(s, src, dst):
    for x in (s["k"], s["v"], s["bounds"]):
        if x is not None:
            x = _by_page(x, s)
            x[:, dst] = x[:, src]


def _fork(s):
    ps, b, dev = s["case"]["page"], s["case"]["batch"], s["lens"].device
    lens, par, row = s["lens"].long(), s["parents"].long(), s["rows"].long()
    full, part = lens // ps, lens % ps
    fresh = (part > 0).long()
    place = s["free_start"].long() + torch.cumsum(fresh, 0) - fresh
    page = s["free"].long()[place.clamp(max=s["free"].numel() - 1)]
    col = torch.arange(s["table"].shape[1], device=dev)[None]
    theirs = s["table"].long()[par]
    mine = torch.where(col < full[:, None], theirs, s["table"].long()[row])
    last = (col == full[:, None]) & (part > 0)[:, None]
    mine = torch.where(last, page[:, None], mine)
    s["table"][row] = mine.to(torch.int32)
    spare = torch.zeros(s["n_pages"] + 1, dtype=torch.int64, device=dev)
    spare.index_add_(0, torch.where(col < full[:, None], theirs, s["n_pages"]).flatten(), torch.ones_like(theirs).flatten())
    s["shares"] += spare[:-1].to(torch.int32)
    s["free_end"][:] = s["free_start"] + fresh.sum()
    tok = torch.arange(s["tokens"].shape[1], device=dev)[None]
    s["tokens"][row] = torch.where(tok < lens[:, None], mine[:, tok[0] // ps] * ps + tok % ps, s["tokens"].long()[row]).to(torch.int32)
    n = sum(s["part"])
    if n:
        e = torch.repeat_interleave(torch.arange(b, device=dev), part, output_size=n)
        off = torch.arange(n, device=dev) - (torch.cumsum(part, 0) - part)[e]
        old = theirs.gather(1, full[:, None])[:, 0]
        for x in (s["k"], s["v"]):
            x[:, page[e] * ps + off] = x[:, old[e] * ps + off]
        if s["bounds"] is not None:
            has = torch.repeat_interleave(torch.arange(b, device=dev), fresh, output_size=sum(p > 0 for p in s["part"]))
            s["bounds"][:, page[has]] = s["bounds"][:, old[has]]


def _release(s):
    ps, dev, n = s["case"]["page"], s["lens"].device, s["n_pages"]
    row = s["rows"].long()
    lo, hi = (s["keep"].long() + ps - 1) // ps, (s["lens"].long() + ps - 1) // ps
    col = torch.arange(s["table"].shape[1], device=dev)[None]
    out = (col >= lo[:, None]) & (col < hi[:, None])
    theirs = s["table"].long()[row]
    drop = torch.zeros(n + 1, dtype=torch.int64, device=dev)
    drop.index_add_(0, torch.where(out, theirs, n).flatten(), torch.ones_like(theirs).flatten())
    left = s["shares"].long() - drop[:n]
    gone = left < 0
    start = s["free_start"].long()
    m = gone.sum()
    room = s["free"].numel()
    place = torch.where(gone, start - m + torch.cumsum(gone, 0) - 1, room)
    free = torch.cat([s["free"], s["free"][:1]])
    free[place] = torch.arange(n, device=dev, dtype=torch.int32)
    s["free"][:] = free[:room]
    s["free_end"][:] = (start - m).to(torch.int32)
    s["shares"][:] = left.clamp(min=0)
    s["table"][row] = torch.where(out, -1, theirs).to(torch.int32)


def _compact(s):
    ps, n, dev = s["case"]["page"], s["n_pages"], s["lens"].device
    start = 5                                   # the free list's place
    free = torch.zeros(n, dtype=torch.bool, device=dev)
    free[s["free"][start:].long()] = True
    used = n - (s["free"].numel() - start)
    src = used + torch.nonzero(~free[used:])[:, 0]
    dst = torch.nonzero(free[:used])[:, 0]
    _copy(s, src, dst)
    to = torch.arange(n, device=dev)
    to[src] = dst
    s["shares"][dst] = s["shares"][src]
    s["shares"][src] = 0
    s["remap"][:] = to
    s["free_out"][start:] = torch.arange(used, n, device=dev)
    t, k = s["table"].long(), s["tokens"].long()
    s["table"][:] = torch.where(t >= 0, to[t.clamp(min=0)], t)
    s["tokens"][:] = torch.where(k >= 0, to[k.clamp(min=0) // ps] * ps + k % ps, k)


def _chunk(s):
    c, ps = s["case"], s["case"]["page"]
    kv, d = c["kv_heads"], c["head_dim"]
    o = torch.empty_like(s["q"])
    at = 0
    for i, (n, m) in enumerate(zip(s["ctx"], s["new"])):
        if not m:
            continue
        page = s["table"].long()[s["rows"][i].long(), :-(-n // ps)]
        slot = (page[:, None] * ps + torch.arange(ps, device=page.device)).flatten()[:n]
        k, v = (x[0][slot].float().transpose(0, 1) for x in (s["k"], s["v"]))                        # [kv, n, d]
        q = s["q"][at:at + m].float().view(m, kv, -1, d).permute(1, 2, 0, 3)                          # [kv, g, m, d]
        w = q @ k[:, None].transpose(-1, -2) / math.sqrt(d)
        if c["causal"]:
            p = torch.arange(n, device=page.device)
            w = w.masked_fill(p > n - m + torch.arange(m, device=page.device)[:, None], -torch.inf)
        if n:
            w = torch.exp(w - w.amax(-1, keepdim=True))
        o[at:at + m] = ((w @ v[:, None]) / w.sum(-1, keepdim=True).clamp(min=1e-37)).permute(2, 0, 1, 3).reshape(m, -1, d).to(o.dtype)
        at += m
    return o


def run(s):
    c, op = s["case"], s["case"]["op"]
    if own:
        import paged_kv_cache_loc_gb300 as pkv
    if op in ("fork", "release", "compact"):    # each pass begins with the same counts (and, where pages are given up, tables)
        s["shares"].copy_(s["shares0"])
    if op == "copy":
        if own:
            pkv.copy_pages(s["cache"], c["page"], s["src"], s["dst"], page_bounds=s["bounds"])
        else:
            _copy(s, s["src"].long(), s["dst"].long())
        return {k: s[k] for k in ("k", "v", "bounds")}
    if op == "fork":
        if own:
            pkv.fork_requests(s["cache"], s["table"], c["page"], s["parents"], s["shares"], s["free"], s["free_start"], s["free_end"],
                              page_bounds=s["bounds"])
        else:
            _fork(s)
        return {k: s[k] for k in ("k", "v", "bounds", "table", "tokens", "shares", "free_end")}
    if op == "release":
        s["table"].copy_(s["table0"])
        if own:
            pkv.release_pages(s["cache"], s["table"], c["page"], s["shares"], s["free"], s["free_start"], s["free_end"], s["keep"])
        else:
            _release(s)
        return {k: s[k] for k in ("table", "shares", "free", "free_end")}
    if op == "compact":
        if own:
            pkv.compact_pages(s["cache"], s["table"], c["page"], s["shares"], s["free"], s["free_start"], s["remap"], free_out=s["free_out"],
                              page_bounds=s["bounds"], workspace=s["ws"])
        else:
            _compact(s)
        return {k: s[k] for k in ("k", "v", "bounds", "table", "tokens", "shares", "remap", "free_out")}
    if own:
        return {"o": pkv.paged_chunk(s["cache"], 0, s["table"], c["page"], s["q"], s["max_q"], causal=c["causal"], workspace=s["ws"])}
    return {"o": _chunk(s)}


def work(case):
    """Bytes: each input row read once and each output written once."""
    op, ps, b, kv, d = case["op"], case["page"], case["batch"], case["kv_heads"], case["head_dim"]
    eb = 4 if case["dtype"] == "f32" else 2
    row = kv * d * eb
    ctx, new = _lengths(case)
    bounds = 2 * row if case["bounds"] else 0
    if op == "copy":
        return {"bytes": case["moves"] * (8 + case["layers"] * 2 * (2 * ps * row + bounds)), "flops": 0}
    if op == "fork":
        full, part = ctx // ps, ctx % ps
        moved = case["layers"] * 2 * (int(part.sum()) * 2 * row + int((part > 0).sum()) * bounds)
        return {"bytes": moved + 12 * b + int(full.sum()) * 16 + int((part > 0).sum()) * 8 + int(ctx.sum()) * 4, "flops": 0}
    if op == "release":
        given = int((-(-ctx // ps) - -(-(ctx - new) // ps)).sum())
        return {"bytes": 12 * b + given * 16, "flops": 0}
    if op == "compact":
        used = case["pages"] // 2 + case["moves"] // 2
        width = max(1, min(-(-case["ctx_hi"] // ps), -(-used // b)))
        return {"bytes": case["moves"] * case["layers"] * 2 * (2 * ps * row + bounds) + 4 * case["pages"] + 8 * (case["pages"] - used)
                + 4 * (b + 3) * (width + 1) * (1 + ps), "flops": 0}
    if case["causal"]:
        pairs = int((new * (ctx - new) + new * (new + 1) // 2).sum())
    else:          # the lengths meet in an order that depends on the seed: their means
        pairs = int(new.sum()) * int(ctx.sum()) // b
    return {"bytes": int(ctx.sum()) * 2 * row + int(-(-ctx // ps).sum()) * 4 + int(new.sum()) * 2 * case["heads"] * d * eb,
            "flops": 4 * d * case["heads"] * pairs}


# ---------------------------------------------------------------------------
# the definitions in 64 bits, entry by entry
# ---------------------------------------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    op, ps, layers = case["op"], case["page"], case["layers"]
    if op == "release":
        return None   # whole numbers alone
    if op != "chunk":
        moved = []    # (first slot, to, slots, page, to)
        if op == "copy":
            moved = [(i * ps, j * ps, ps, i, j) for i, j in zip(s["src"].tolist(), s["dst"].tolist())]
        elif op == "fork":
            table, take = s["table"].cpu().numpy(), iter(s["free"].tolist()[5:])
            for p, n in zip(s["parents"].tolist(), s["lens"].tolist()):
                if n % ps:
                    i, j = int(table[p, n // ps]), next(take)
                    moved.append((i * ps, j * ps, n % ps, i, j))
        else:
            free = set(s["free"].tolist()[5:])
            used = [i for i in range(s["n_pages"]) if i not in free]
            late = [i for i in used if i >= len(used)]
            holes = sorted(i for i in free if i < len(used))
            moved = [(i * ps, j * ps, ps, i, j) for i, j in zip(late, holes)]
        for i, j, n, p, r in moved:
            for x in (s["k"], s["v"]):
                x[:, j:j + n].copy_(x[:, i:i + n])
            if s["bounds"] is not None:
                s["bounds"][:, r].copy_(s["bounds"][:, p])
        got = {k: s[k] for k in ("k", "v", "bounds")}
        if op == "fork":
            got.update(table=None, tokens=None, shares=None, free_end=None)
        if op == "compact":
            got.update(table=None, tokens=None, shares=None, remap=None, free_out=None)
        return got
    kv, d, g = case["kv_heads"], case["head_dim"], case["heads"] // case["kv_heads"]
    o = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    table, at = s["table"].cpu().numpy(), 0
    for i, (n, m) in enumerate(zip(s["ctx"], s["new"])):
        pos = np.arange(n)
        slot = torch.from_numpy(table[int(s["rows"][i]), pos // ps].astype(np.int64) * ps + pos % ps).cuda()
        for h in range(kv if n and m else 0):
            k, v = s["k"][0, slot, h].double(), s["v"][0, slot, h].double()
            for r0 in range(0, m, 512):        # rows that fit
                q = s["q"][at + r0:at + min(m, r0 + 512), h * g:(h + 1) * g].double()
                w = torch.einsum("qgd,nd->gqn", q, k) / math.sqrt(d)
                if case["causal"]:
                    seen = n - m + r0 + torch.arange(q.shape[0], device="cuda")
                    w = torch.where(torch.arange(n, device="cuda")[None] <= seen[:, None], w, -torch.inf)
                o[at + r0:at + r0 + q.shape[0], h * g:(h + 1) * g] = torch.einsum("gqn,nd->qgd", torch.softmax(w, -1), v)
        at += m
    return {"o": o}
