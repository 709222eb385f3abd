"""The paged K/V cache operators, for measuring: append, decode attention, prompt attention and the
operations on pages, each in its plain form (elementary torch operations in 32 bits) and through the
framework's entry points.

Cache layout: k, v [n_layers][n_pages][n_kv_heads][page_size][head_dim], table int32
[max_seqs][max_pages] (page of each page_size positions of a sequence, -1 = none), refs int32
[n_pages] (sequences that hold the page, 0 = free).
"""
import math

import torch

own = False

DTYPES = {"fp16": torch.float16, "bf16": torch.bfloat16}


def listed():
    return [
        # one sequence generating alone on a small model (16 heads x 64, 2048 cached): latency
        dict(name="decode_one", op="decode", lanes=1, heads=16, kv=16, hd=64, page=16, dtype="fp16", lo=2049, hi=2049),
        # a full batch of equal long contexts, every head with K and V of its own (16 x 128, 32 lanes, 4096 cached)
        dict(name="decode_batch", op="decode", lanes=32, heads=16, kv=16, hd=128, page=64, dtype="fp16", lo=4097, hi=4097),
        # a serving batch: grouped heads, lengths from nothing cached to 8192
        dict(name="decode_ragged", op="decode", lanes=48, heads=32, kv=8, hd=128, page=16, dtype="bf16", lo=0, hi=8192),
        # one very long context on few K/V heads: only its length can fill the GPU
        dict(name="decode_long", op="decode", lanes=1, heads=16, kv=2, hd=128, page=32, dtype="bf16", lo=60001, hi=60001),
        # a short first prompt of a small model: latency
        dict(name="prompt_one", op="prompt", lanes=1, heads=4, kv=4, hd=64, page=16, dtype="fp16", lo=130, hi=130, cached=0),
        # a batch of prompts of different lengths, packed
        dict(name="prompt_packed", op="prompt", lanes=24, heads=16, kv=4, hd=128, page=32, dtype="fp16", lo=1, hi=2048, cached=0),
        # one long prompt
        dict(name="prompt_long", op="prompt", lanes=1, heads=16, kv=4, hd=128, page=64, dtype="bf16", lo=16384, hi=16384, cached=0),
        # chunked prefill: a chunk of each prompt over what the cache already holds
        dict(name="prompt_chunk", op="prompt", lanes=4, heads=32, kv=8, hd=128, page=16, dtype="bf16", lo=300, hi=512, cached=8192),
        # the new token's K and V of a serving batch: latency
        dict(name="append_token", op="append", lanes=48, kv=8, hd=128, page=16, dtype="bf16", lo=1, hi=1),
        # the K and V of a batch of packed prompts
        dict(name="append_prompt", op="append", lanes=24, kv=8, hd=128, page=16, dtype="fp16", lo=1, hi=2048),
        # parallel sampling: prompts forked, each fork given room for its next token (the shared last page copied), the
        # forks of the step before freed
        dict(name="pages_fork", op="fork", lanes=12, copies=4, layers=8, kv=8, hd=128, page=16, dtype="bf16", lo=100, hi=4000, n_pages=4096),
        # a fragmented pool compacted after most of its sequences ended
        dict(name="pages_compact", op="compact", lanes=48, layers=4, kv=8, hd=128, page=16, dtype="fp16", lo=500, hi=2700, n_pages=8192),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["decode", "decode", "prompt", "prompt", "append", "fork", "compact"])
    c = dict(op=op, kv=rng.choice([1, 2, 3, 4, 8, 16]), hd=rng.choice([64, 128]), page=rng.choice([16, 32, 64, 128]),
             dtype=rng.choice(["fp16", "bf16"]))
    if op == "decode":
        c.update(lanes=_log(rng, 1, 64), heads=c["kv"] * rng.choice([1, 2, 4, 5, 8]))
        most = max(2, min(60000, (1 << 28) // (c["lanes"] * c["kv"] * c["hd"])))
        c["hi"] = _log(rng, 2, most)
        c["lo"] = rng.choice([0, 1, c["hi"] // 2, c["hi"]])
    elif op == "prompt":
        c.update(lanes=_log(rng, 1, 24), heads=c["kv"] * rng.choice([1, 2, 3, 4, 8]), cached=rng.choice([0, 0, _log(rng, 1, 8000)]))
        room = (1 << 31) // (c["lanes"] * c["heads"])  # padded scores of the plain form
        c["cached"] = min(c["cached"], room // 64)
        most = max(2, int(min(8192, (math.sqrt(c["cached"] ** 2 + 4 * room) - c["cached"]) / 2)))
        c["hi"] = _log(rng, 2, most)
        c["lo"] = rng.choice([1, (c["hi"] + 1) // 2, c["hi"]])
    elif op == "append":
        c.update(lanes=_log(rng, 1, 64), hi=_log(rng, 1, 1024))
        c["lo"] = rng.choice([1, c["hi"]])
    elif op == "fork":
        c.update(lanes=_log(rng, 1, 12), copies=rng.randint(1, 4), layers=rng.randint(1, 8))
        most = (1 << 29) // (c["layers"] * c["kv"] * c["hd"] * c["lanes"])
        c["hi"] = _log(rng, 20, max(20, min(4000, most)))
        c["lo"] = rng.choice([1, c["hi"] // 2])
    else:
        c.update(lanes=_log(rng, 2, 48), layers=rng.randint(1, 4))
        c["n_pages"] = max(100, min(8192, (1 << 29) // (c["layers"] * c["kv"] * c["page"] * c["hd"]) - rng.randint(0, 50)))
        most = c["n_pages"] // c["lanes"] * c["page"]
        c["hi"] = _log(rng, min(40, most), most)
        c["lo"] = c["hi"] // 4
    return c


def _lengths(case, seed):
    """The lanes' lengths, spread over [lo, hi], the ends among them."""
    g = torch.Generator().manual_seed(seed * 2 + 1)
    n, lo, hi = case["lanes"], case["lo"], case["hi"]
    v = torch.randint(lo, hi + 1, (n,), generator=g).tolist()
    v[0] = hi
    if n > 1:
        v[-1] = lo
    if n > 2:
        v[1] = min(max(1, lo), hi)
    return v


def _pages_of(n, page):
    return -(-n // page)


def prepare(case, seed):
    c, lens = dict(case), _lengths(case, 0)  # the amount of work does not go by the seed
    g = torch.Generator(device="cuda").manual_seed(seed)
    cpu = torch.Generator().manual_seed(seed)
    dt, op, page = DTYPES[c["dtype"]], c["op"], c["page"]
    cached = c.get("cached", 0)
    kv_len = [n + (cached - 37 * (b % 5) if cached > 200 else cached) for b, n in enumerate(lens)]
    if op == "append":
        start = [13 * b % 40 for b in range(c["lanes"])]
        kv_len = [n + s for n, s in zip(lens, start)]
    need = [_pages_of(n, page) for n in kv_len]
    max_pages = max(1, max(need)) + (1 if op == "fork" else 0)
    max_seqs = c["lanes"] * (1 + c.get("copies", 0))
    n_pages = c.get("n_pages", sum(need) + c["lanes"] * c.get("copies", 0) + 8)
    layers = c.get("layers", 1)
    shape = (layers, n_pages, c["kv"], page, c["hd"])
    st = {"case": c, "kv_len": kv_len, "max_len": max(kv_len)}
    st["k"] = torch.empty(shape, dtype=dt, device="cuda").normal_(generator=g)
    st["v"] = torch.empty(shape, dtype=dt, device="cuda").normal_(generator=g)
    # pages in a random order, as after some time of serving
    order = torch.randperm(n_pages, generator=cpu)[: sum(need)].to(torch.int32)
    table = torch.full((max_seqs, max_pages), -1, dtype=torch.int32)
    refs = torch.zeros(n_pages, dtype=torch.int32)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = order[at: at + n]
        at += n
    refs[order.long()] = 1
    st["table"], st["refs"] = table.cuda(), refs.cuda()
    heads, lanes = c.get("heads", c["kv"]), c["lanes"]
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    st["len"] = i32(kv_len)
    cu = [0]
    for n in lens:
        cu.append(cu[-1] + n)
    if op == "decode":
        st["q"] = torch.empty((lanes, heads, c["hd"]), dtype=dt, device="cuda").normal_(generator=g)
        st["out"] = torch.zeros_like(st["q"])
    elif op == "prompt":
        st["q"] = torch.empty((cu[-1], heads, c["hd"]), dtype=dt, device="cuda").normal_(generator=g)
        st["out"] = torch.zeros_like(st["q"])
        st["cu"], st["max_q"] = i32(cu), max(lens)
    elif op == "append":
        st["rows_k"] = torch.empty((cu[-1], c["kv"], c["hd"]), dtype=dt, device="cuda").normal_(generator=g)
        st["rows_v"] = torch.empty((cu[-1], c["kv"], c["hd"]), dtype=dt, device="cuda").normal_(generator=g)
        st["cu"], st["start"] = i32(cu), i32(start)
    elif op == "fork":
        src = [b for b in range(lanes) for _ in range(c["copies"])]
        st["src"], st["dst"] = i32(src), i32([lanes + i for i in range(len(src))])
        st["fork_len"], st["one"] = i32([kv_len[b] for b in src]), i32([1] * len(src))
    else:
        st["table0"], st["refs0"] = st["table"].clone(), st["refs"].clone()
        st["n_live"] = i32([0])
    if own:
        import store_kv_attention_b200 as tl
        desc = tl.PagedDesc(n_layers=layers, n_pages=n_pages, page_size=page, n_kv_heads=c["kv"], head_dim=c["hd"],
                            max_seqs=max_seqs, max_pages=max_pages, dtype=tl.TL_KV_FP16 if dt == torch.float16 else tl.TL_KV_BF16)
        st["cache"] = tl.PagedCache(desc, n_heads=heads, n_lanes=max_seqs, k=st["k"], v=st["v"], table=st["table"],
                                    refs=st["refs"])
    return st


# ---------------------------------------------------------------- the plain forms
def _gathered(st, pool, n):
    """Rows 0 .. n-1 of every lane from the pages of layer 0: fp32 [lanes, kv, n, hd], zero where a lane has no such row."""
    lanes, page = st["len"].numel(), pool.shape[3]
    pages = st["table"][:lanes, : max(1, _pages_of(n, page))].clamp(min=0).long()
    x = pool[0][pages].transpose(1, 2).flatten(2, 3)[:, :, :n].float()
    alive = torch.arange(x.shape[2], device=x.device)[None, :] < st["len"][:, None]
    return torch.where(alive[:, None, :, None], x, 0.0), alive


def _attend(s, mask, v):
    """softmax of s over its last axis where mask holds, times v; zero where a row attends nothing."""
    s = s.masked_fill_(~mask, -math.inf)
    m = s.amax(-1, keepdim=True)
    p = s.sub_(torch.where(torch.isfinite(m), m, 0.0)).exp_()
    total = p.sum(-1, keepdim=True)
    return torch.matmul(p, v) / torch.where(total > 0, total, 1.0)


def _plain_decode(st):
    q = st["q"].float()
    lanes, heads, hd = q.shape
    k, alive = _gathered(st, st["k"], st["max_len"])
    v, _ = _gathered(st, st["v"], st["max_len"])
    kv = k.shape[1]
    s = torch.matmul(q.view(lanes, kv, heads // kv, hd) * hd ** -0.5, k.transpose(2, 3))
    return _attend(s, alive[:, None, None, :], v).reshape(lanes, heads, hd).to(st["q"].dtype)


def _plain_prompt(st):
    q, cu, n = st["q"], st["cu"].long(), st["max_q"]
    total, heads, hd = q.shape
    k, alive = _gathered(st, st["k"], st["max_len"])
    v, _ = _gathered(st, st["v"], st["max_len"])
    lanes, kv = k.shape[:2]
    i = torch.arange(n, device=q.device)
    inside = i[None, :] < (cu[1:] - cu[:-1])[:, None]
    at = torch.where(inside, cu[:-1, None] + i[None, :], 0)
    x = q.float()[at].view(lanes, n, kv, heads // kv, hd).permute(0, 2, 3, 1, 4).reshape(lanes, kv, -1, hd)
    s = torch.matmul(x * hd ** -0.5, k.transpose(2, 3)).view(lanes, kv, heads // kv, n, -1)
    place = (st["len"].long() - (cu[1:] - cu[:-1]))[:, None] + i[None, :]
    mask = (torch.arange(s.shape[-1], device=q.device)[None, None, :] <= place[:, :, None]) & alive[:, None, :]
    o = _attend(s, mask[:, None, None], v[:, :, None]).permute(0, 3, 1, 2, 4).reshape(lanes, n, heads, hd)
    return o[inside].to(q.dtype)


def _plain_append(st):
    cu, rows = st["cu"].long(), st["rows_k"].shape[0]
    r = torch.arange(rows, device=cu.device)
    lane = torch.searchsorted(cu, r, right=True) - 1
    pos = st["start"].long()[lane] + r - cu[lane]
    page = st["k"].shape[3]
    p = st["table"][lane, pos // page].long()
    st["k"][0, p, :, pos % page] = st["rows_k"]
    st["v"][0, p, :, pos % page] = st["rows_v"]
    return st["k"], st["v"]


def _plain_fork(st):
    table, refs, page = st["table"], st["refs"], st["k"].shape[3]
    src, dst, n = st["src"].long(), st["dst"].long(), st["fork_len"].long()
    # free the forks of the step before
    old = table[dst]
    refs.index_add_(0, old[old >= 0].long(), -torch.ones_like(old[old >= 0]))
    # fork: the pages of the first n tokens are shared
    held = torch.arange(table.shape[1], device=table.device)[None, :] < ((n + page - 1) // page)[:, None]
    new = torch.where(held, table[src], -1)
    refs.index_add_(0, new[held].long(), torch.ones_like(new[held]))
    # reserve one token: the page it falls into, if none or shared, becomes the lowest free page, with its rows
    j = (n // page)[:, None]
    was = new.gather(1, j)[:, 0]
    need = (was < 0) | (refs[was.clamp(min=0).long()] > 1)
    free = torch.nonzero(refs == 0)[:, 0].to(torch.int32)
    got = free[(torch.cumsum(need, 0) - 1).clamp(min=0)]
    table[dst] = new.scatter(1, j, torch.where(need, got, was)[:, None])
    shared = need & (was >= 0)
    refs.index_add_(0, was[shared].long(), -torch.ones_like(was[shared]))
    refs[got[need].long()] = 1
    a, b = was[shared].long(), got[shared].long()
    st["k"][:, b] = st["k"][:, a]
    st["v"][:, b] = st["v"][:, a]
    return table, refs, st["k"], st["v"]


def _plain_compact(st):
    table, refs = st["table"], st["refs"]
    table.copy_(st["table0"])
    refs.copy_(st["refs0"])
    live = refs > 0
    n = live.sum()
    at = torch.arange(refs.numel(), device=refs.device)
    holes, movers = torch.nonzero(~live & (at < n))[:, 0], torch.nonzero(live & (at >= n))[:, 0]
    st["k"][:, holes] = st["k"][:, movers]
    st["v"][:, holes] = st["v"][:, movers]
    to = at.clone()
    to[movers] = holes
    table.copy_(torch.where(table >= 0, to[table.clamp(min=0).long()].to(torch.int32), table))
    refs[holes] = refs[movers]
    refs[movers] = 0
    st["n_live"].copy_(n[None])
    return table, refs, st["n_live"], st["k"], st["v"]


PLAIN = {"decode": _plain_decode, "prompt": _plain_prompt, "append": _plain_append, "fork": _plain_fork, "compact": _plain_compact}


def run(st):
    op = st["case"]["op"]
    if not own:
        return PLAIN[op](st)
    import store_kv_attention_b200 as tl
    cache = st["cache"]
    if op == "decode":
        tl.paged_attn_decode(cache, 0, st["q"], st["len"], st["out"])
        return st["out"]
    if op == "prompt":
        tl.paged_prompt_attn(cache, 0, st["q"], st["cu"], st["len"], st["out"])
        return st["out"]
    if op == "append":
        tl.paged_append(cache, 0, st["rows_k"], st["rows_v"], st["start"], cu_rows=st["cu"])
        return st["k"], st["v"]
    if op == "fork":
        tl.paged_free(cache, st["dst"])
        tl.paged_fork(cache, st["src"], st["dst"], st["fork_len"])
        tl.paged_reserve(cache, st["dst"], st["fork_len"], st["one"])
        return st["table"], st["refs"], st["k"], st["v"]
    st["table"].copy_(st["table0"])
    st["refs"].copy_(st["refs0"])
    tl.paged_compact(cache, st["n_live"])
    return st["table"], st["refs"], st["n_live"], st["k"], st["v"]


# ---------------------------------------------------------------- what a pass cannot do without
def work(case):
    c, lens = case, _lengths(case, 0)
    row = c["kv"] * c["hd"] * 2  # bytes of one position's K (or V)
    cached = c.get("cached", 0)
    kv_len = [n + (cached - 37 * (b % 5) if cached > 200 else cached) for b, n in enumerate(lens)]
    if c["op"] == "decode":
        return {"bytes": 2 * row * sum(kv_len) + 4 * c["lanes"] * c["heads"] * c["hd"], "flops": 4 * c["heads"] * c["hd"] * sum(kv_len)}
    if c["op"] == "prompt":
        pairs = sum(q * (k - q) + q * (q + 1) // 2 for q, k in zip(lens, kv_len))
        return {"bytes": 2 * row * sum(kv_len) + 4 * sum(lens) * c["heads"] * c["hd"], "flops": 4 * c["heads"] * c["hd"] * pairs}
    if c["op"] == "append":
        return {"bytes": 4 * row * sum(lens), "flops": 0}
    table = 4 * sum(_pages_of(n, c["page"]) for n in lens)
    if c["op"] == "fork":
        ends = sum(n % c["page"] > 0 for n in lens)
        return {"bytes": c["copies"] * (ends * 4 * row * c["page"] * c["layers"] + 4 * table), "flops": 0}
    # movers of a random live set: live pages at or above the live count
    live = table // 4
    moved = int(live * (1 - live / c["n_pages"]))
    return {"bytes": 4 * row * c["page"] * c["layers"] * moved + 2 * table + 4 * c["n_pages"], "flops": 0}


# ---------------------------------------------------------------- from the definitions, in 64 bits
def exact(case, seed):
    was = globals()["own"]
    globals()["own"] = False
    try:
        st = prepare(case, seed)
    finally:
        globals()["own"] = was
    op, page, hd = case["op"], case["page"], case["hd"]
    k, v, table = st["k"], st["v"], st["table"].cpu()
    if op in ("decode", "prompt"):
        out = torch.zeros(st["q"].shape, dtype=torch.float64, device="cuda")
        cu = st["cu"].tolist() if op == "prompt" else list(range(case["lanes"] + 1))
        group = case["heads"] // case["kv"]
        for b, n in enumerate(st["kv_len"]):
            nq = cu[b + 1] - cu[b]
            if n <= 0 or nq <= 0:
                continue
            ids = [int(p) for p in table[b, : _pages_of(n, page)]]
            for h in range(case["heads"]):
                kk = torch.cat([k[0, p, h // group] for p in ids])[:n].double()
                vv = torch.cat([v[0, p, h // group] for p in ids])[:n].double()
                for lo in range(0, nq, 2048):
                    q = st["q"][cu[b] + lo: min(cu[b] + lo + 2048, cu[b + 1]), h].double()
                    s = q @ kk.T / math.sqrt(hd)
                    if op == "prompt":
                        i = torch.arange(lo, lo + q.shape[0], device="cuda")
                        late = torch.arange(n, device="cuda")[None, :] > (n - nq + i)[:, None]
                        s[late] = -math.inf
                    out[cu[b] + lo: cu[b] + lo + q.shape[0], h] = torch.softmax(s, -1).nan_to_num(0.0) @ vv
        return out
    if op == "append":
        cu, start = st["cu"].tolist(), st["start"].tolist()
        for b in range(case["lanes"]):
            n, r = cu[b + 1] - cu[b], 0
            while r < n:
                pos = start[b] + r
                m = min(n - r, page - pos % page)
                p = int(table[b, pos // page])
                for pool, rows in ((k, st["rows_k"]), (v, st["rows_v"])):
                    pool[0, p, :, pos % page: pos % page + m] = rows[cu[b] + r: cu[b] + r + m].transpose(0, 1)
                r += m
        return k.double(), v.double()
    refs = st["refs"].cpu()
    if op == "fork":
        rows = list(zip(st["src"].tolist(), st["dst"].tolist(), st["fork_len"].tolist()))
        for s, d, n in rows:
            for j in range(_pages_of(n, page)):
                table[d, j] = table[s, j]
                refs[int(table[s, j])] += 1
        held, free = refs.clone(), iter([p for p, r in enumerate(refs.tolist()) if r == 0])
        for s, d, n in rows:
            p = int(table[d, n // page])
            if p < 0 or held[p] > 1:
                to = next(free)
                table[d, n // page], refs[to] = to, 1
                if p >= 0:
                    refs[p] -= 1
                    k[:, to] = k[:, p]
                    v[:, to] = v[:, p]
        return table.long(), refs.long(), k.double(), v.double()
    live = [p for p, r in enumerate(refs.tolist()) if r > 0]
    n = len(live)
    to = dict(zip([p for p in live if p >= n], [p for p in range(n) if refs[p] == 0]))
    for p, h in to.items():
        k[:, h] = k[:, p]
        v[:, h] = v[:, p]
        refs[h], refs[p] = int(refs[p]), 0
    table = torch.tensor([[to.get(p, p) for p in r] for r in table.tolist()])
    return table, refs.long(), torch.tensor([n]), k.double(), v.double()
