"""Cases of the key-value cache's operators: the page plan, the write into the cache, the attention that reads it.

``own`` False computes the plain forms in torch; True calls the library (``lib.PagedCache``). A case is one pass of one operator:

  plan    block tables and slot maps for a step, from the requests' lengths and the free pages
  write   RMSNorm per head and rotary embedding of q and k, and the append of k and v by slot
  attend  attention of one new token of each request over its pages, with an optional sigmoid gate on the output

The lengths of a case are a fixed set that the seed only puts in another order, so its work does not depend on the seed.
"""
import math

import torch

own = False

E4M3_MAX = 448.0
EPS = 1e-6
THETA = 1e7
GAMMA_OFFSET = 1.0          # the norm's weight is offset + gamma

DTYPES = {"f16": torch.float16, "bf16": torch.bfloat16, "e4m3": torch.float8_e4m3fn}


def listed():
    return [
        # a decode step of a small server: eight requests, one new token each, a page now and then
        dict(name="plan decode 8", op="plan", requests=8, shortest=20, longest=900, prompts=0, prompt=0, done=0, page=16,
             spare=64, padding=0),
        # continuous batching: most requests decode, some finish and give their pages back, a few new prompts come in
        dict(name="plan mixed 301", op="plan", requests=301, shortest=1, longest=6000, prompts=9, prompt=700, done=23, page=16,
             spare=4096, padding=37),
        # a large pool that runs out of pages: many prompts at once, the last ones refused
        dict(name="plan prompts 2048", op="plan", requests=2048, shortest=1, longest=2500, prompts=500, prompt=1000, done=100,
             page=32, spare=7000, padding=0),
        # one token's q, k and v of the gated attention layer
        dict(name="write decode 1", op="write", tokens=1, heads=16, kv_heads=2, dim=256, rope=64, page=16, act="f16",
             cache="f16", padding=0),
        # a decode step of a full server into an 8-bit cache, a few rows of it padding
        dict(name="write decode 250 e4m3", op="write", tokens=250, heads=16, kv_heads=2, dim=256, rope=64, page=16, act="bf16",
             cache="e4m3", padding=6),
        # a long prompt's rows, rotary over the whole head
        dict(name="write prompt 8192", op="write", tokens=8192, heads=32, kv_heads=8, dim=128, rope=128, page=64, act="bf16",
             cache="bf16", padding=0),
        # the smallest step: one request early in its answer
        dict(name="attend 1 x 130", op="attend", requests=1, shortest=130, longest=130, empty=0, heads=16, kv_heads=2, dim=256,
             page=16, act="f16", cache="f16", gate=True),
        # one request with a very long context
        dict(name="attend 1 x 131072", op="attend", requests=1, shortest=131072, longest=131072, empty=0, heads=16, kv_heads=2,
             dim=256, page=16, act="f16", cache="f16", gate=True),
        # sixteen independent tokens, lengths spread over two decades
        dict(name="attend 16 ragged", op="attend", requests=16, shortest=61, longest=8191, empty=0, heads=16, kv_heads=2,
             dim=256, page=16, act="f16", cache="f16", gate=True),
        # a full server: large batch, long contexts, some slots without a request
        dict(name="attend 128 ragged", op="attend", requests=128, shortest=512, longest=16000, empty=5, heads=16, kv_heads=2,
             dim=256, page=16, act="f16", cache="f16", gate=True),
        # a larger batch over an 8-bit cache
        dict(name="attend 256 e4m3", op="attend", requests=256, shortest=300, longest=5000, empty=0, heads=16, kv_heads=2,
             dim=256, page=32, act="bf16", cache="e4m3", gate=True),
        # heads of 128, four query heads to a key head, no gate
        dict(name="attend 61 x 128-wide", op="attend", requests=61, shortest=1, longest=9000, empty=1, heads=32, kv_heads=8,
             dim=128, page=64, act="bf16", cache="bf16", gate=False),
    ]


#: (query heads, key-value heads) of the drawn cases: groups of 1 to 32 query heads, odd ones among them.
HEADS = [(16, 2), (32, 8), (8, 8), (16, 1), (14, 2), (9, 3), (5, 1), (32, 1), (6, 6), (64, 4)]


def _spread(rng, low, high):
    return min(high, max(low, int(round(math.exp(rng.uniform(math.log(low), math.log(high + 1)))))))


def draw(rng):
    op = rng.choice(["plan", "write", "attend", "attend"])
    page = rng.choice([16, 32, 64, 128])
    if op == "plan":
        n = _spread(rng, 1, 2048)
        shortest = _spread(rng, 1, 500)
        longest = _spread(rng, shortest, 6000)
        prompts = rng.randrange(0, 1 + n // 4)
        prompt = _spread(rng, 1, 1000)
        done = rng.randrange(0, 1 + n // 8)
        return dict(op="plan", requests=n, shortest=shortest, longest=longest, prompts=prompts, prompt=prompt, done=done,
                    page=page, spare=_spread(rng, 1, 2 * n + 2 * prompts * (1 + prompt // page)), padding=rng.randrange(0, 64))
    heads, kv_heads = rng.choice(HEADS)
    dim = rng.choice([64, 128, 256])
    act = rng.choice(["f16", "bf16"])
    cache = rng.choice([act, "e4m3"])
    if op == "write":
        # at most the bytes of the largest listed case
        tokens = _spread(rng, 1, min(8192, 8192 * 192 * 128 // ((4 * heads + 8 * kv_heads) * dim)))
        return dict(op="write", tokens=tokens, heads=heads, kv_heads=kv_heads, dim=dim, rope=rng.choice([0, dim // 4, dim // 2, dim]),
                    page=page, act=act, cache=cache, padding=rng.randrange(0, 1 + tokens // 8))
    # up to about half the bytes of the largest listed case
    most = 300_000 * 1024 // (kv_heads * dim * 2)
    n = _spread(rng, 1, 256)
    longest = _spread(rng, 1, max(1, min(131072, most // n)))
    return dict(op="attend", requests=n, shortest=_spread(rng, 1, longest), longest=longest, empty=rng.randrange(0, 1 + n // 4),
                heads=heads, kv_heads=kv_heads, dim=dim, page=page, act=act, cache=cache, gate=rng.random() < 0.5)


def _lengths(case):
    """The case's lengths, from the shortest to the longest in equal ratios; the last `empty` ones are 0."""
    n, lo, hi = case["requests"], case["shortest"], case["longest"]
    v = [int(round(lo * (hi / lo) ** (i / max(1, n - 1)))) for i in range(n)]
    v[0], v[-1] = lo, hi
    k = case.get("empty", 0)
    return [0] * k + v[k:]


def _new_tokens(case):
    """Cached and new tokens of each request of a plan: prompts have none cached, -1 ends a request."""
    cached = _lengths(case)
    new = [1] * case["requests"]
    for i in range(case["prompts"]):
        cached[4 * i] = 0
        new[4 * i] = 1 + (case["prompt"] - 1) * (i + 1) // case["prompts"]
    for i in range(case["done"]):
        new[4 * i + 1 if 4 * i + 1 < len(new) else -1] = -1
    return cached, new


def _pages(tokens, page):
    return -(-tokens // page)


def _tables(lengths, page, width, n_pages, gen, dev):
    """A table of pages for the lengths, -1 where a request has none, and the pages that are left."""
    order = torch.randperm(n_pages, generator=gen, device=dev).to(torch.int32)
    held = (lengths + page - 1) // page
    before = held.cumsum(0) - held
    j = torch.arange(width, device=dev)
    at = before[:, None] + j
    return torch.where(j < held[:, None], order[at.clamp(max=n_pages - 1)], -1), order, held


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)
    op, page = case["op"], case["page"]
    s = {"case": case}

    def randn(*shape, dtype, gain=1.0):
        return (torch.randn(*shape, generator=gen, device=dev, dtype=torch.float32 if dtype == torch.float8_e4m3fn else dtype) * gain).to(dtype)

    if op == "plan":
        cached, new = _new_tokens(case)
        order = torch.randperm(len(cached), generator=gen, device=dev)
        cached = torch.tensor(cached, device=dev)[order]
        new = torch.tensor(new, device=dev)[order]
        held = sum(_pages(c, page) for c in _new_tokens(case)[0])
        n_pages = held + case["spare"]
        width = max(_pages(c + max(n, 0), page) for c, n in zip(*_new_tokens(case))) + 2
        tables, pages, _ = _tables(cached, page, width, n_pages, gen, dev)
        # the free pages lie in a ring, from `head` on; the rest of the ring holds what was there before
        head = int(seed * 7919 % n_pages)
        at = (head + torch.arange(case["spare"], device=dev)) % n_pages
        ring = torch.full((n_pages,), -1, dtype=torch.int32, device=dev)
        ring[at] = pages[held:]
        rows = sum(max(n, 0) for n in _new_tokens(case)[1]) + case["padding"]
        s |= dict(lengths=cached.to(torch.int32), new=new.to(torch.int32), tables=tables.contiguous(), ring=ring, rows=rows,
                  n_pages=n_pages, free=torch.tensor([head, case["spare"], 0], dtype=torch.int32, device=dev))
        return s
    act, cache = DTYPES[case["act"]], DTYPES[case["cache"]]
    heads, kv_heads, dim = case["heads"], case["kv_heads"], case["dim"]
    if cache == torch.float8_e4m3fn:  # the largest value of a head on the type's largest
        s["k_scale"] = (torch.rand(kv_heads, generator=gen, device=dev) + 0.5) * (6.0 / E4M3_MAX)
        s["v_scale"] = (torch.rand(kv_heads, generator=gen, device=dev) + 0.5) * (6.0 / E4M3_MAX)
    else:
        s["k_scale"] = s["v_scale"] = None
    if op == "write":
        tokens = case["tokens"]
        n_pages = _pages(tokens, page) + 3
        # q, k and v as the projections leave them: views of one matrix, the gate beside each query head
        x = randn(tokens, 2 * heads + 2 * kv_heads, dim, dtype=act, gain=1.5)
        s["q"] = x[:, : 2 * heads].view(tokens, heads, 2, dim)[:, :, 0]
        s["k"], s["v"] = x[:, 2 * heads: 2 * heads + kv_heads], x[:, 2 * heads + kv_heads:]
        s["q_gamma"], s["k_gamma"] = randn(dim, dtype=act, gain=0.2), randn(dim, dtype=act, gain=0.2)
        # the last page belongs to nobody; rows of padding have slot -1
        slots = torch.randperm((n_pages - 1) * page, generator=gen, device=dev)[:tokens].to(torch.int32)
        slots[tokens - case["padding"]:] = -1
        s["slots"] = slots[torch.randperm(tokens, generator=gen, device=dev)].contiguous()
        s["positions"] = torch.randint(0, 262144, (tokens,), generator=gen, device=dev, dtype=torch.int32)
        s["k_cache"] = randn(n_pages, kv_heads, page, dim, dtype=cache)
        s["v_cache"] = randn(n_pages, kv_heads, page, dim, dtype=cache)
        s["n_pages"] = n_pages
        return s
    lengths = torch.tensor(_lengths(case), device=dev)[torch.randperm(case["requests"], generator=gen, device=dev)]
    total = sum(_pages(n, page) for n in _lengths(case))
    n_pages, width = total + 1, _pages(case["longest"], page) + 1
    s["tables"], _, held = _tables(lengths, page, width, n_pages, gen, dev)
    s["tables"] = s["tables"].contiguous()
    gain = 16.0 if cache == torch.float8_e4m3fn else 1.0
    s["k_cache"] = torch.empty(n_pages, kv_heads, page, dim, device=dev, dtype=cache)
    s["v_cache"] = torch.empty(n_pages, kv_heads, page, dim, device=dev, dtype=cache)
    for pool in (s["k_cache"], s["v_cache"]):
        if cache == torch.float8_e4m3fn:
            pool.copy_(torch.randn(pool.shape, generator=gen, device=dev, dtype=torch.float16).mul_(gain))
        else:
            pool.normal_(generator=gen)
    # what lies past a request's end in its last page was never written: NaN (the pool's last page is nobody's)
    last = s["tables"].gather(1, (held - 1).clamp(min=0)[:, None])[:, 0]
    last = torch.where(held > 0, last, n_pages - 1).long()
    past = torch.arange(page, device=dev) >= (lengths - (held - 1).clamp(min=0) * page)[:, None]
    for pool in (s["k_cache"], s["v_cache"]):
        raw, nan = (pool.view(torch.uint8), 0x7F) if cache == torch.float8_e4m3fn else (pool.view(torch.int16), 0x7FFF)
        raw[last] = raw[last].masked_fill(past[:, None, :, None], nan)
    s["q"] = randn(case["requests"], heads, dim, dtype=act, gain=2.0)
    s["gate"] = randn(case["requests"], heads, dim, dtype=act) if case["gate"] else None
    s["lengths"] = lengths.to(torch.int32)
    s["n_pages"] = n_pages
    return s


_caches = {}


def _cache(s):
    """The program's handle for a shape: made once, as a server makes it when it loads a model."""
    c = s["case"]
    key = (c["op"], c.get("heads", 16), c.get("kv_heads", 2), c.get("dim", 256), c["page"], c.get("act", "f16"), c.get("cache", "f16"),
           c.get("rope", 0), s["n_pages"], c.get("requests", 1), s["tables"].shape[1] if "tables" in s else 1)
    if key not in _caches:
        from w4a16_top_mixture_gb300 import lib
        _caches[key] = lib.PagedCache(n_heads=key[1], n_kv_heads=key[2], head_dim=key[3], page_size=key[4], dtype=key[5],
                                      cache_dtype=key[6], rope_dim=key[7], rope_theta=THETA, gamma_offset=GAMMA_OFFSET, eps=EPS,
                                      n_pages=key[8], max_requests=key[9], max_pages=key[10])
    return _caches[key]


def run(s):
    op = s["case"]["op"]
    if own:
        c = _cache(s)
        if op == "plan":
            p = c.plan(s["lengths"], s["new"], s["tables"], s["ring"], s["free"], s["rows"])
            return dict(slots=p.slots, positions=p.positions, starts=p.starts, lengths=p.lengths, free=p.free_state,
                        tables=s["tables"], ring=s["ring"])
        if op == "write":
            q = c.write(s["q"], s["k"], s["v"], s["positions"], s["slots"], s["k_cache"], s["v_cache"], q_gamma=s["q_gamma"],
                        k_gamma=s["k_gamma"], k_scale=s["k_scale"], v_scale=s["v_scale"])
            return dict(q=q, k_cache=s["k_cache"], v_cache=s["v_cache"])
        return c.attend(s["q"], s["tables"], s["lengths"], s["k_cache"], s["v_cache"], gate=s["gate"], k_scale=s["k_scale"],
                        v_scale=s["v_scale"])
    return {"plan": _plan, "write": _write, "attend": _attend}[op](s)


def _plan(s):
    page, ring, tables, rows, n_pages = s["case"]["page"], s["ring"], s["tables"], s["rows"], s["n_pages"]
    dev, width, n_ring = tables.device, tables.shape[1], ring.shape[0]
    cached, new = s["lengths"].long(), s["new"].long()
    head, count = s["free"][0].long(), s["free"][1].long()
    done = new < 0
    n = new.clamp(min=0)
    ends = n.cumsum(0)
    starts = ends - n
    own_pages = (cached + page - 1) // page
    want = (cached + n + page - 1) // page
    fits = ~done & (want <= width) & (ends <= rows)
    need = torch.where(fits, want - own_pages, 0)
    upto = need.cumsum(0)
    ok = fits & ((need == 0) | (upto <= count))
    before = upto - need
    # pages that finished requests give back, to the ring's end
    back = torch.where(done, own_pages, 0)
    back_upto = back.cumsum(0)
    given = back_upto[-1]
    off = (torch.arange(n_ring, device=dev) - head - count) % n_ring
    giver = torch.searchsorted(back_upto, off, right=True).clamp(max=len(back) - 1)
    j = (off - (back_upto - back)[giver]).clamp(0, width - 1)
    ring_out = torch.where(off < given, tables[giver, j], ring)
    # pages that admitted requests take, from its head
    col = torch.arange(width, device=dev)
    fresh = ring[(head + before[:, None] + col - own_pages[:, None]) % n_ring]
    tables.copy_(torch.where(ok[:, None] & (col >= own_pages[:, None]) & (col < want[:, None]), fresh, tables))
    ring.copy_(ring_out)
    taken = torch.where(ok, need, 0).sum()
    row = torch.arange(rows, device=dev)
    of = torch.searchsorted(ends, row, right=True)
    inside = of < len(n)
    of = of.clamp(max=len(n) - 1)
    held = inside & ok[of]
    pos = torch.where(held, cached[of] + row - starts[of], 0)
    page_id = tables[of, (pos // page).clamp(max=width - 1)].long()
    slots = torch.where(held & (page_id >= 0) & (page_id < n_pages), page_id * page + pos % page, -1)
    i32 = torch.int32
    return dict(slots=slots.to(i32), positions=pos.to(i32), starts=torch.cat([starts, ends[-1:]]).to(i32),
                lengths=torch.where(done, 0, torch.where(ok, cached + n, cached)).to(i32),
                free=torch.stack([(head + taken) % n_ring, count - taken + given, (~ok & ~done).sum()]).to(i32), tables=tables, ring=ring)


def _norm_rope(x, gamma, positions, rope):
    x = x.float()
    y = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS) * (GAMMA_OFFSET + gamma.float())
    if not rope:
        return y
    half = rope // 2
    freq = THETA ** (-2.0 * torch.arange(half, dtype=torch.float64, device=x.device) / rope)
    angle = positions.double()[:, None, None] * freq
    cos, sin = angle.cos().float(), angle.sin().float()
    a, b = y[..., :half], y[..., half:rope]
    return torch.cat([a * cos - b * sin, b * cos + a * sin, y[..., rope:]], -1)


def _write(s):
    case = s["case"]
    page, rope = case["page"], case["rope"]
    q = _norm_rope(s["q"], s["q_gamma"], s["positions"], rope).to(s["q"].dtype)
    rows = {"k": _norm_rope(s["k"], s["k_gamma"], s["positions"], rope), "v": s["v"].float()}
    # rows without a slot put back what the pool's last slot, which is nobody's, holds
    slot = s["slots"].long()
    held = slot >= 0
    slot = torch.where(held, slot, s["n_pages"] * page - 1)
    at, off = slot // page, slot % page
    for name, x in rows.items():
        pool, scale = s[name + "_cache"], s[name + "_scale"]
        if scale is not None:
            x = (x / scale[:, None]).clamp(-E4M3_MAX, E4M3_MAX)
        raw = pool.view(torch.uint8) if pool.dtype == torch.float8_e4m3fn else pool
        raw[at, :, off] = torch.where(held[:, None, None], x.to(pool.dtype).view(raw.dtype), raw[at, :, off])
    return dict(q=q, k_cache=s["k_cache"], v_cache=s["v_cache"])


def _attend(s):
    case = s["case"]
    n, heads, kv_heads, dim, page = case["requests"], case["heads"], case["kv_heads"], case["dim"], case["page"]
    width = _pages(case["longest"], page)
    at = s["tables"][:, :width].long().clamp(min=0)
    valid = torch.arange(width * page, device=at.device) < s["lengths"][:, None]          # [n, L]

    def gathered(pool):  # [n, kv, L, dim]
        raw = pool.view(torch.uint8) if pool.dtype == torch.float8_e4m3fn else pool
        return raw[at].view(pool.dtype).transpose(1, 2).reshape(n, kv_heads, width * page, dim).float()

    q = s["q"].float().view(n, kv_heads, heads // kv_heads, dim)
    score = q @ gathered(s["k_cache"]).transpose(-1, -2) * dim ** -0.5
    if s["k_scale"] is not None:
        score = score * s["k_scale"][:, None, None]
    score = torch.where(valid[:, None, None], score, -torch.inf)
    top = score.amax(-1, keepdim=True)
    e = torch.exp(score - torch.where(top == -torch.inf, 0.0, top))
    v = torch.where(valid[:, None, :, None], gathered(s["v_cache"]), 0.0)
    if s["v_scale"] is not None:
        v = v * s["v_scale"][:, None, None]
    out = e @ v / e.sum(-1, keepdim=True)
    out = torch.where(valid[:, :1, None, None], out, 0.0).view(n, heads, dim)
    if s["gate"] is not None:
        out = out * torch.sigmoid(s["gate"].float())
    return out.to(s["q"].dtype)


def work(case):
    page = case["page"]
    if case["op"] == "plan":
        cached, new = _new_tokens(case)
        rows = sum(max(x, 0) for x in new) + case["padding"]
        back = sum(_pages(c, page) for c, x in zip(cached, new) if x < 0)
        need = sum(_pages(c + x, page) - _pages(c, page) for c, x in zip(cached, new) if x >= 0)
        return {"bytes": 16 * case["requests"] + 8 * rows + 8 * (back + min(need, case["spare"])), "flops": 0}
    heads, kv_heads, dim = case["heads"], case["kv_heads"], case["dim"]
    size, c_size = 2, 1 if case["cache"] == "e4m3" else 2
    if case["op"] == "write":
        tokens, held = case["tokens"], case["tokens"] - case["padding"]
        return {"bytes": tokens * 2 * heads * dim * size + held * 2 * kv_heads * dim * (size + c_size) + 8 * tokens + 2 * dim * size,
                "flops": tokens * (heads + kv_heads) * dim * 8}
    lengths = _lengths(case)
    tokens, rows = sum(lengths), case["requests"] * heads * dim * size
    return {"bytes": tokens * kv_heads * dim * 2 * c_size + rows * (3 if case["gate"] else 2) + 4 * sum(_pages(x, page) for x in lengths)
            + 4 * case["requests"], "flops": 4 * heads * dim * tokens}


def exact(case, seed):
    if case["op"] == "plan":
        return None                      # whole numbers
    s = prepare(case, seed)
    dim, kv_heads, page = case["dim"], case["kv_heads"], case["page"]
    if case["op"] == "write":
        half = case["rope"] // 2
        turn = torch.ones(case["tokens"], 1, dim // 2, dtype=torch.complex128, device="cuda")
        if half:
            freq = torch.exp(torch.arange(half, dtype=torch.float64, device="cuda") * (-math.log(THETA) / half))
            angle = torch.outer(s["positions"].to(torch.float64), freq)
            turn = torch.polar(torch.ones_like(angle), angle)[:, None]

        def rotated(x, gamma):
            x = x.to(torch.float64)
            x = x / (x.pow(2).sum(-1, keepdim=True) / dim + EPS).sqrt() * (gamma.to(torch.float64) + GAMMA_OFFSET)
            if half:
                z = torch.complex(x[..., :half].contiguous(), x[..., half: 2 * half].contiguous()) * turn
                x = torch.cat((z.real, z.imag, x[..., 2 * half:]), dim=-1)
            return x

        out = {"q": rotated(s["q"], s["q_gamma"])}
        slots = s["slots"].tolist()
        take = [t for t, p in enumerate(slots) if p >= 0]
        put = torch.tensor([slots[t] for t in take], dtype=torch.int64, device="cuda")
        for name, x in (("k", rotated(s["k"], s["k_gamma"])), ("v", s["v"].to(torch.float64))):
            flat = s[name + "_cache"].to(torch.float64).permute(0, 2, 1, 3).reshape(-1, kv_heads, dim).clone()
            x = x[torch.tensor(take, dtype=torch.int64, device="cuda")]
            if s[name + "_scale"] is not None:
                x = (x / s[name + "_scale"].to(torch.float64).view(1, -1, 1)).clamp(-E4M3_MAX, E4M3_MAX)
            flat[put] = x
            out[name + "_cache"] = flat.view(s["n_pages"], page, kv_heads, dim).permute(0, 2, 1, 3).contiguous()
        return out
    q = s["q"].to(torch.float64)
    out = torch.zeros(q.shape, dtype=torch.float64, device="cuda")
    group = case["heads"] // kv_heads
    for b, length in enumerate(s["lengths"].tolist()):
        if not length:
            continue
        ids = s["tables"][b, : _pages(length, page)].to(torch.int64)
        for h in range(kv_heads):
            k = s["k_cache"][:, h].view(torch.uint8 if case["cache"] == "e4m3" else torch.int16)[ids].view(DTYPES[case["cache"]])
            v = s["v_cache"][:, h].view(torch.uint8 if case["cache"] == "e4m3" else torch.int16)[ids].view(DTYPES[case["cache"]])
            k, v = (x.reshape(-1, dim)[:length].to(torch.float64) for x in (k, v))
            if s["k_scale"] is not None:
                k, v = k * s["k_scale"][h].to(torch.float64), v * s["v_scale"][h].to(torch.float64)
            mine = slice(h * group, (h + 1) * group)
            out[b, mine] = torch.softmax(q[b, mine] @ k.T / math.sqrt(dim), dim=-1) @ v
    if s["gate"] is not None:
        out = out / (1 + torch.exp(-s["gate"].to(torch.float64)))
    return out
