"""Cases of the key-value cache's operators for steps that bring several tokens of a request: drafted trees and chains,
what of them is kept, and requests that share pages.

``own`` False computes the plain forms in torch; True calls the library (``lib.PagedCache``). A case is one pass of one operator:

  tree    ancestor masks and positions of drafted trees, from each token's parent
  attend  attention of each request's new tokens over its pages: all older tokens, and those of the new ones its mask names
  keep    the accepted tokens move up in every layer's pools, the pages behind them are given back
  fork    further requests over the same tokens: full pages are shared, the last one is copied in every layer's pools

The lengths of a case are a fixed set that the seed only puts in another order, so its work does not depend on the seed.
"""
import math

import numpy as np
import torch

own = False

E4M3_MAX = 448.0
DTYPES = {"f16": torch.float16, "bf16": torch.bfloat16, "e4m3": torch.float8_e4m3fn}


def listed():
    wide = dict(heads=16, kv_heads=2, dim=256, page=16)
    return [
        # one user's step with a small tree
        dict(name="tree 1 x 26", op="tree", requests=1, fewest=26, nodes=26, longest=900, refused=0, padding=0),
        # a full server, trees of up to 60 tokens, some requests refused for want of pages
        dict(name="tree 256 x 60", op="tree", requests=256, fewest=4, nodes=60, longest=6000, refused=3, padding=31),
        # the smallest step: one request early in its answer, five drafted tokens
        dict(name="attend 1 x 130, 5 new", op="attend", requests=1, shortest=130, longest=130, empty=0, refused=0, fewest=5,
             nodes=5, tree=True, act="f16", cache="f16", gate=True, padding=0, **wide),
        # one request with a very long context, a chain of five
        dict(name="attend 1 x 131072, chain of 5", op="attend", requests=1, shortest=131072, longest=131072, empty=0, refused=0,
             fewest=5, nodes=5, tree=False, act="f16", cache="f16", gate=True, padding=0, **wide),
        # sixteen independent answers, trees of 64 tokens, lengths over two decades
        dict(name="attend 16 ragged, trees of 64", op="attend", requests=16, shortest=80, longest=8191, empty=0, refused=0,
             fewest=64, nodes=64, tree=True, act="f16", cache="f16", gate=True, padding=0, **wide),
        # a full server over an 8-bit cache: small trees, some slots empty, one request refused, a few rows of padding
        dict(name="attend 128 e4m3, trees to 16", op="attend", requests=128, shortest=512, longest=9000, empty=4, refused=1,
             fewest=5, nodes=16, tree=True, act="bf16", cache="e4m3", gate=True, padding=9, **wide),
        # prompts that enter the cache in chunks of 256 tokens, heads of 128
        dict(name="attend 24 chunks of 256", op="attend", requests=24, shortest=256, longest=8192, empty=0, refused=0, fewest=256,
             nodes=256, tree=False, act="bf16", cache="bf16", gate=False, padding=0, heads=32, kv_heads=8, dim=128, page=64),
        # one request, a chain whose first tokens were right: nothing moves, its last pages go
        dict(name="keep 1 chain", op="keep", requests=1, shortest=500, longest=500, fewest=5, nodes=5, accept=3, chain=True, done=0,
             shared=0, pools=20, kv_heads=2, dim=256, page=16, cache="f16", spare=64),
        # a full server after a step with trees of up to 60: a path of each tree stays, in the ten attention layers' pools
        dict(name="keep 256 trees", op="keep", requests=256, shortest=20, longest=900, fewest=16, nodes=60, accept=8, chain=False,
             done=9, shared=0, pools=20, kv_heads=2, dim=256, page=16, cache="f16", spare=4096),
        # requests that share prompts, over an 8-bit cache; many of them end and give shared pages back
        dict(name="keep 301 shared", op="keep", requests=301, shortest=300, longest=3000, fewest=2, nodes=16, accept=5, chain=False,
             done=60, shared=100, pools=8, kv_heads=8, dim=128, page=32, cache="e4m3", spare=2000),
        # one prompt, four answers
        dict(name="fork 1 to 3", op="fork", sources=1, copies=3, shortest=700, longest=700, pools=20, kv_heads=2, dim=256, page=16,
             cache="f16", spare=64),
        # beams of a full server: 32 requests to four each, pages of 64 tokens
        dict(name="fork 32 to 96", op="fork", sources=32, copies=3, shortest=100, longest=9000, pools=20, kv_heads=2, dim=256,
             page=64, cache="bf16", spare=500),
    ]


#: (query heads, key-value heads) of the drawn cases: groups of 1 to 32 query heads, odd ones among them.
HEADS = [(16, 2), (32, 8), (8, 8), (16, 1), (14, 2), (9, 3), (5, 1), (32, 1), (6, 6), (64, 4)]


def _spread(rng, low, high):
    high = max(low, high)
    return min(high, max(low, int(round(math.exp(rng.uniform(math.log(low), math.log(high + 1)))))))


def draw(rng):
    op = rng.choice(["tree", "attend", "attend", "attend", "keep", "fork"])
    page = rng.choice([16, 32, 64, 128])
    nodes = _spread(rng, 1, 256)
    fewest = _spread(rng, 1, nodes)
    if op == "tree":
        n = _spread(rng, 1, min(256, 256 * 60 // nodes))
        return dict(op="tree", requests=n, fewest=fewest, nodes=nodes, longest=_spread(rng, nodes, 6000), refused=rng.randrange(0, 1 + n // 8),
                    padding=rng.randrange(0, 64))
    heads, kv_heads = rng.choice(HEADS)
    dim = rng.choice([64, 128, 256])
    act = rng.choice(["f16", "bf16"])
    cache = rng.choice([act, "e4m3"])
    if op == "attend":
        # up to about half the work of the largest listed case: of its products, and of the bytes of the longest one
        tokens = min(300_000 * 1024 // (kv_heads * dim * 2), 24 * 1200 * 256 * 32 * 128 // (nodes * heads * dim))
        n = _spread(rng, 1, max(1, min(128, tokens // nodes)))
        longest = _spread(rng, nodes, min(131072, tokens // n))
        return dict(op="attend", requests=n, shortest=_spread(rng, nodes, longest), longest=longest, empty=rng.randrange(0, 1 + n // 6),
                    refused=rng.randrange(0, 1 + n // 8), fewest=fewest, nodes=nodes, tree=rng.random() < 0.7, heads=heads, kv_heads=kv_heads,
                    dim=dim, page=page, act=act, cache=cache, gate=rng.random() < 0.5, padding=rng.randrange(0, 32))
    pools = rng.randrange(1, 21)
    if op == "keep":
        nodes = min(nodes, 64)
        fewest = min(fewest, nodes)
        n = _spread(rng, 1, min(301, 256 * 60 // nodes))
        longest = _spread(rng, 1, min(3000, 200_000 * 1024 // (n * kv_heads * dim * 2)))
        return dict(op="keep", requests=n, shortest=_spread(rng, 1, longest), longest=longest, fewest=fewest, nodes=nodes,
                    accept=rng.randrange(0, 1 + min(fewest, 8)), chain=rng.random() < 0.3, done=rng.randrange(0, 1 + n // 4),
                    shared=rng.randrange(0, 1 + n // 3), pools=pools, kv_heads=kv_heads, dim=dim, page=page, cache=cache,
                    spare=_spread(rng, 1, 4 * n))
    sources = _spread(rng, 1, 32)
    longest = _spread(rng, 1, min(9000, 200_000 * 1024 // (sources * kv_heads * dim * 2)))
    return dict(op="fork", sources=sources, copies=rng.randrange(1, 4), shortest=_spread(rng, 1, longest), longest=longest, pools=pools,
                kv_heads=kv_heads, dim=dim, page=page, cache=cache, spare=_spread(rng, 1, 4 * sources))


def _pages(tokens, page):
    return -(-tokens // page)


def _ratios(lo, hi, n):
    """n whole numbers from lo to hi in equal ratios."""
    v = [int(round(lo * (hi / lo) ** (i / max(1, n - 1)))) for i in range(n)]
    v[0], v[-1] = lo, hi
    return v


def _requests(case):
    """(tokens in the cache, new ones among them, whether the plan refused the new ones) of each request, the longest last.
    Empty requests come first, then the refused ones, whose new tokens have rows but are not in the cache."""
    n = case["requests"]
    lengths = _ratios(case.get("shortest", case["nodes"]), case["longest"], n)
    span = case["nodes"] - case["fewest"] + 1
    new = [case["nodes"] - 7 * (n - 1 - i) % span for i in range(n)]
    out = []
    for i in range(n):
        if i < case.get("empty", 0):
            out.append((0, 0, False))
        else:
            out.append((max(lengths[i], new[i]), new[i], i < case.get("empty", 0) + case["refused"]))
    return out


def _drafts(case):
    """(older tokens, new tokens, kept: -1 where the request ends) of each request of a keep."""
    n = case["requests"]
    older = _ratios(case["shortest"], case["longest"], n)
    span = case["nodes"] - case["fewest"] + 1
    new = [case["nodes"] - 7 * (n - 1 - i) % span for i in range(n)]
    # of a tree the first token is not on the path, so that all that stays moves
    most = [min(case["accept"], m if case["chain"] else m - 1) for m in new]
    kept = [max(0, m - i % 3) if n > 1 else m for i, m in enumerate(most)]
    for i in range(case["done"]):
        kept[4 * i + 1 if 4 * i + 1 < n else i % n] = -1
    return older, new, kept


def _tables(lengths, page, width, n_pages, gen, dev):
    """A table of pages for the lengths, -1 where a request has none, and the pages in the order they were given out."""
    order = torch.randperm(n_pages, generator=gen, device=dev).to(torch.int32)
    held = (lengths + page - 1) // page
    before = held.cumsum(0) - held
    j = torch.arange(width, device=dev)
    at = before[:, None] + j
    return torch.where(j < held[:, None], order[at.clamp(max=n_pages - 1)], -1).contiguous(), order, held


def _ring(free, n_pages, seed, dev):
    """The free pages in a ring, from a head that the seed chooses, and its state."""
    head = int(seed * 7919 % n_pages)
    ring = torch.full((n_pages,), -1, dtype=torch.int32, device=dev)
    ring[(head + torch.arange(len(free), device=dev)) % n_pages] = free
    return ring, torch.tensor([head, len(free), 0], dtype=torch.int32, device=dev)


def _pool_values(shape, dtype, gen, dev):
    if dtype == torch.float8_e4m3fn:
        return torch.randn(shape, generator=gen, device=dev, dtype=torch.float16).mul_(16.0).to(dtype)
    return torch.empty(shape, device=dev, dtype=dtype).normal_(generator=gen)


def _shuffled(rows, gen, dev):
    t = torch.tensor(rows, device=dev)
    return t[torch.randperm(len(rows), generator=gen, device=dev)]


def _prepare_new(s, case, gen, dev):
    """Lengths, rows and parents of requests with new tokens."""
    r = _shuffled([(a, b, int(c)) for a, b, c in _requests(case)], gen, dev)
    lengths, new, refused = r[:, 0], r[:, 1], r[:, 2] > 0
    starts = torch.cat([new.new_zeros(1), new.cumsum(0)])
    rows = sum(b for _, b, _ in _requests(case)) + case["padding"]
    row = torch.arange(rows, device=dev)
    of = torch.searchsorted(starts[1:].contiguous(), row, right=True)
    inside = of < len(new)
    of = of.clamp(max=len(new) - 1)
    i = row - starts[of]
    # a parent among the last few tokens before it, or none: bushy trees with paths of some length
    back = 1 + (torch.rand(rows, generator=gen, device=dev) ** 2 * 6).long()
    s["parents"] = torch.where(inside, (i - back).clamp(min=-1), -1).to(torch.int32)
    s["lengths"], s["starts"] = lengths.to(torch.int32), starts.to(torch.int32)
    s["rows"], s["words"] = rows, _pages(case["nodes"], 64)
    return lengths, new, refused, of, inside, i


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)
    op, s = case["op"], {"case": case}
    if op == "tree":
        lengths, new, refused, of, inside, i = _prepare_new(s, case, gen, dev)
        slots = torch.randint(0, 1 << 20, (s["rows"],), generator=gen, device=dev)
        s["slots"] = torch.where(inside & ~refused[of], slots, -1).to(torch.int32)
        return s
    page, dim, kv_heads, cache = case["page"], case["dim"], case["kv_heads"], DTYPES[case["cache"]]
    if op == "attend":
        act, heads = DTYPES[case["act"]], case["heads"]
        lengths, new, refused, of, inside, i = _prepare_new(s, case, gen, dev)
        total = sum(_pages(a, page) for a, _, _ in _requests(case))
        n_pages, width = total + 1, max(1, _pages(max(a for a, _, _ in _requests(case)), page)) + 1
        s["tables"], _, held = _tables(lengths, page, width, n_pages, gen, dev)
        pos = (lengths - new)[of] + i
        at = s["tables"].long()[of, (pos // page).clamp(0, width - 1)]
        s["slots"] = torch.where(inside & ~refused[of], at * page + pos % page, -1).to(torch.int32)
        s["k_cache"], s["v_cache"] = (_pool_values((n_pages, kv_heads, page, dim), cache, gen, dev) for _ in range(2))
        # what lies past a request's end in its last page was never written: NaN
        have = held > 0
        last = s["tables"].long().gather(1, (held - 1).clamp(min=0)[:, None])[:, 0][have]
        past = (torch.arange(page, device=dev) >= (lengths - (held - 1) * page)[:, None])[have]
        for pool in (s["k_cache"], s["v_cache"]):
            raw, nan = (pool.view(torch.uint8), 0x7F) if cache == torch.float8_e4m3fn else (pool.view(torch.int16), 0x7FFF)
            raw[last] = raw[last].masked_fill(past[:, None, :, None], nan)
        if cache == torch.float8_e4m3fn:
            s["k_scale"], s["v_scale"] = ((torch.rand(kv_heads, generator=gen, device=dev) + 0.5) * (1.0 / 16.0) for _ in range(2))
        else:
            s["k_scale"] = s["v_scale"] = None
        s["q"] = (torch.randn(s["rows"], heads, dim, generator=gen, device=dev) * 2.0).to(act)
        s["gate"] = torch.randn(s["rows"], heads, dim, generator=gen, device=dev).to(act) if case["gate"] else None
        s["out"] = torch.zeros_like(s["q"])           # rows of padding stay as they are
        s["n_pages"], s["slots"] = n_pages, s["slots"].contiguous()
        s["masks"] = _tree(s)["masks"] if case["tree"] else None
        return s
    if op == "keep":
        older, new, kept = (torch.tensor(v, device=dev) for v in _drafts(case))
        order = torch.randperm(len(new), generator=gen, device=dev)
        older, new, kept = older[order], new[order], kept[order]
        lengths = older + new
        a, b, _ = _drafts(case)
        total = sum(_pages(x + y, page) for x, y in zip(a, b))
        n_pages, width = total + case["spare"], max(_pages(x + y, page) for x, y in zip(a, b)) + 2
        s["tables"], pages, held = _tables(lengths, page, width, n_pages, gen, dev)
        free = pages[total:]
        s["refs"] = None
        if case["shared"]:
            # request 2i + 1 begins with the full pages of request 2i's older tokens, as far as its own reach
            refs = torch.zeros(n_pages, dtype=torch.int32, device=dev)
            pairs = min(case["shared"], len(new) // 2)
            one, two = s["tables"][0: 2 * pairs: 2], s["tables"][1: 2 * pairs: 2]
            both = torch.minimum(older[0: 2 * pairs: 2], older[1: 2 * pairs: 2]) // page
            common = torch.arange(width, device=dev) < both[:, None]
            free = torch.cat([free, two[common]])
            refs[one[common].long()] = 1
            s["tables"][1: 2 * pairs: 2] = torch.where(common, one, two)
            s["refs"] = refs
        s["ring"], s["free"] = _ring(free, n_pages, seed, dev)
        s["path"] = None
        if not case["chain"]:
            # ascending, the first token of a tree not among them
            score = torch.rand(len(new), case["nodes"], generator=gen, device=dev)
            j = torch.arange(case["nodes"], device=dev)
            score = torch.where((j >= 1) & (j < new[:, None]), score, 2.0)
            take = score.argsort(1)[:, : max(1, case["accept"])]
            take = torch.where(torch.arange(take.shape[1], device=dev) < kept[:, None], take, case["nodes"]).sort(1)[0]
            s["path"] = take.to(torch.int32).contiguous()
        s["starts"] = torch.cat([new.new_zeros(1), new.cumsum(0)]).to(torch.int32)
        s["counts"], s["lengths"] = kept.to(torch.int32), lengths.to(torch.int32)
        s["slots"] = None
    else:
        older = _ratios(case["shortest"], case["longest"], case["sources"])
        n, copies = case["sources"], case["copies"]
        order = torch.randperm(n * (1 + copies), generator=gen, device=dev)
        lengths = torch.zeros(n * (1 + copies), dtype=torch.long, device=dev)
        lengths[order[:n]] = torch.tensor(older, device=dev)
        total = sum(_pages(x, page) for x in older)
        n_pages, width = total + case["spare"], max(_pages(x, page) for x in older) + 2
        s["tables"], pages, _ = _tables(lengths, page, width, n_pages, gen, dev)
        s["ring"], s["free"] = _ring(pages[total:], n_pages, seed, dev)
        s["refs"] = torch.zeros(n_pages, dtype=torch.int32, device=dev)
        s["src"], s["dst"] = order[:n].repeat(copies).to(torch.int32), order[n:].to(torch.int32).contiguous()
        s["lengths"] = lengths.to(torch.int32)
    s["pools"] = [_pool_values((n_pages, kv_heads, page, dim), cache, gen, dev) for _ in range(case["pools"])]
    s["n_pages"] = n_pages
    if own:
        s["pool_list"] = _cache(s).pools(s["pools"])      # the addresses of the layers' pools, as a server keeps them
    return s


_caches = {}


def _cache(s):
    """The program's handle for a shape: made once, as a server makes it when it loads a model."""
    c = s["case"]
    B, width = (s["tables"].shape if "tables" in s else (s["lengths"].shape[0], 1 + c["longest"] // 16))
    key = (c.get("heads", c.get("kv_heads", 2)), c.get("kv_heads", 2), c.get("dim", 256), c.get("page", 16), s.get("n_pages", 1),
           B, width, c.get("act", "bf16" if c.get("cache") == "bf16" else "f16"), c.get("cache", "f16"), c.get("nodes", 1))
    if key not in _caches:
        from w4a16_top_mixture_gb300 import lib
        _caches[key] = lib.PagedCache(n_heads=key[0], n_kv_heads=key[1], head_dim=key[2], page_size=key[3], n_pages=key[4],
                                      max_requests=key[5], max_pages=key[6], dtype=key[7], cache_dtype=key[8], max_new=key[9])
    return _caches[key]


def run(s):
    op = s["case"]["op"]
    if own:
        c = _cache(s)
        if op == "tree":
            t = c.tree(s["parents"], s["starts"], s["lengths"], slots=s["slots"])
            return dict(masks=t.masks, positions=t.positions)
        if op == "attend":
            return c.attend_tree(s["q"], s["starts"], s["tables"], s["lengths"], s["k_cache"], s["v_cache"], masks=s["masks"],
                                 slots=s["slots"], gate=s["gate"], k_scale=s["k_scale"], v_scale=s["v_scale"], out=s["out"])
        if op == "keep":
            r = c.keep(s["counts"], s["lengths"], s["tables"], s["ring"], s["free"], s["pool_list"], starts=s["starts"],
                       path=s["path"], refs=s["refs"])
        else:
            r = c.fork(s["src"], s["dst"], s["lengths"], s["tables"], s["ring"], s["free"], s["refs"], s["pool_list"])
        return dict(lengths=r.lengths, free=r.free_state, tables=s["tables"], ring=s["ring"], refs=s["refs"], pools=s["pools"])
    return {"tree": _tree, "attend": _attend, "keep": _keep, "fork": _fork}[op](s)


def _rows_of(s):
    """Each row's request, its place among the request's new tokens, and whether it has a token in the cache."""
    starts, slots = s["starts"].long(), s["slots"].long()
    row = torch.arange(s["rows"], device=starts.device)
    of = torch.searchsorted(starts[1:].contiguous(), row, right=True)
    inside = of < len(starts) - 1
    of = of.clamp(max=len(starts) - 2)
    first = slots[starts[of].clamp(max=s["rows"] - 1)]
    return of, row - starts[of], inside & (first >= 0)


def _tree(s):
    starts, lengths, words = s["starts"].long(), s["lengths"].long(), s["words"]
    of, i, held = _rows_of(s)
    parent = torch.where(held, s["parents"].long(), -1)
    seen = (torch.arange(64 * words, device=i.device) == i[:, None]) & held[:, None]
    depth = held.long()
    # each row takes its ancestor's ancestors, and then looks twice as far up
    up = torch.where(parent >= 0, starts[of] + parent, -1)
    for _ in range(8):
        at = up.clamp(min=0)
        seen = seen | (seen[at] & (up >= 0)[:, None])
        depth = depth + torch.where(up >= 0, depth[at], 0)
        up = torch.where(up >= 0, up[at], -1)
    masks = (seen.view(-1, words, 64).long() << torch.arange(64, device=i.device)).sum(-1)
    new = starts[1:] - starts[:-1]
    positions = torch.where(held, (lengths - new)[of] + depth - 1, 0)
    return dict(masks=masks, positions=positions.to(torch.int32))


def _attend(s):
    case = s["case"]
    heads, kv_heads, dim, page = case["heads"], case["kv_heads"], case["dim"], case["page"]
    starts, lengths, group = s["starts"].long(), s["lengths"].long(), heads // kv_heads
    n, dev = len(lengths), lengths.device
    N = case["nodes"]
    width = max(1, _pages(max(a for a, _, _ in _requests(case)), page))
    at = s["tables"][:, :width].long().clamp(min=0)
    pos = torch.arange(width * page, device=dev)
    i = torch.arange(N, device=dev)
    row = (starts[:-1, None] + i).clamp(max=s["rows"] - 1)                                # [n, N]
    held = (i < (starts[1:] - starts[:-1])[:, None]) & (s["slots"].long()[row[:, :1]] >= 0)
    older = lengths - (starts[1:] - starts[:-1])
    rel = pos - older[:, None]                                                            # [n, L]
    if s["masks"] is None:
        sees = rel[:, None] <= i[:, None]
    else:
        word = s["masks"][row].gather(2, (rel.clamp(0, 64 * s["words"] - 1) // 64)[:, None].expand(n, N, -1))
        sees = (rel[:, None] < 0) | ((word >> (rel.clamp(min=0) % 64)[:, None]) & 1 > 0)
    valid = pos < lengths[:, None]
    sees = sees & valid[:, None] & held[..., None]                                        # [n, N, L]

    def gathered(pool):  # [n, kv, L, dim]
        raw = pool.view(torch.uint8) if pool.dtype == torch.float8_e4m3fn else pool
        return raw[at].view(pool.dtype).transpose(1, 2).reshape(n, kv_heads, width * page, dim).float()

    q = s["q"][row].float().view(n, N, kv_heads, group, dim).transpose(1, 2).reshape(n, kv_heads, N * group, dim)
    score = (q @ gathered(s["k_cache"]).transpose(-1, -2)).view(n, kv_heads, N, group, -1) * dim ** -0.5
    if s["k_scale"] is not None:
        score = score * s["k_scale"][:, None, None, None]
    score = torch.where(sees[:, None, :, None], score, -torch.inf)
    top = score.amax(-1, keepdim=True)
    e = torch.exp(score - torch.where(top == -torch.inf, 0.0, top))
    total = e.sum(-1, keepdim=True)
    v = torch.where(valid[:, None, :, None], gathered(s["v_cache"]), 0.0)
    if s["v_scale"] is not None:
        v = v * s["v_scale"][:, None, None]
    out = (e.view(n, kv_heads, N * group, -1) @ v).view(n, kv_heads, N, group, dim) / torch.where(total == 0, 1.0, total)
    out = out.transpose(1, 2).reshape(n, N, heads, dim)
    if s["gate"] is not None:
        out = out * torch.sigmoid(s["gate"][row].float())
    of, place, _ = _rows_of(s)
    inside = torch.arange(s["rows"], device=dev) < starts[-1]
    out = torch.where(inside[:, None, None], out[of, place.clamp(0, N - 1)].to(s["q"].dtype), s["out"])
    return out


def _move(pools, page, src, dst):
    """Rows of tokens from slots to slots, all of them read before any is written."""
    for pool in pools:
        raw = pool.view(torch.uint8) if pool.dtype == torch.float8_e4m3fn else pool
        raw[dst // page, :, dst % page] = raw[src // page, :, src % page]


def _keep(s):
    page, tables, ring, refs, n_pages = s["case"]["page"], s["tables"], s["ring"], s["refs"], s["n_pages"]
    dev, width, n_ring = tables.device, tables.shape[1], ring.shape[0]
    lengths, starts, counts = s["lengths"].long(), s["starts"].long(), s["counts"].long()
    head, count = s["free"][0].long(), s["free"][1].long()
    older = lengths - (starts[1:] - starts[:-1])
    ended = counts < 0
    k = counts.clamp(min=0)
    new = torch.where(ended, 0, older + k)
    col, b = torch.arange(width, device=dev), torch.arange(len(k), device=dev)
    held, stay = (lengths + page - 1) // page, (new + page - 1) // page
    path = s["path"].long() if s["path"] is not None else torch.arange(max(1, s["case"]["accept"]), device=dev).expand(len(k), -1)
    j = torch.arange(path.shape[1], device=dev)
    moved = (j < k[:, None]) & (path != j)
    some = moved.any(1)
    first = torch.where(some, older + moved.long().argmax(1), torch.where(new % page > 0, new - 1, stay * page)) // page
    # shared pages that would be written, now or by the next token, are replaced by fresh ones
    page_id = tables.long().clamp(min=0)
    if refs is not None:
        own_copy = (refs[page_id] > 0) & (col >= first[:, None]) & (col < stay[:, None]) & ~ended[:, None]
    else:
        own_copy = torch.zeros_like(tables, dtype=torch.bool)
    need = own_copy.sum(1)
    upto = need.cumsum(0)
    ok = (need == 0) | (upto <= count)
    own_copy = own_copy & ok[:, None]
    fresh = ring[(head + (upto - need)[:, None] + own_copy.cumsum(1) - 1) % n_ring]
    tables_out = torch.where(own_copy, fresh, tables)
    new = torch.where(ok, new, lengths)
    # the pages that nobody holds any more, in the order of the first request that gave each back
    leaving = own_copy | (ok[:, None] & (col >= stay[:, None]) & (col < held[:, None]))
    if refs is not None:
        left = refs.index_add(0, page_id.flatten(), -leaving.flatten().to(torch.int32))
        owner = torch.full((n_pages,), len(k), device=dev).scatter_reduce(
            0, page_id.flatten(), torch.where(leaving, b[:, None], len(k)).flatten(), "amin")
        gives = leaving & (left[page_id] < 0) & (owner[page_id] == b[:, None])
        refs.copy_(left.clamp(min=0))
    else:
        gives = leaving
    place = gives.flatten().cumsum(0) - 1
    given = gives.sum().clamp(max=n_ring - count)
    put = gives.flatten() & (place < given)
    ring[((head + count + place) % n_ring)[put]] = tables.flatten()[put]
    taken = torch.where(ok, need, 0).sum()
    # the rows
    p = first[:, None] * page + torch.arange(page + path.shape[1], device=dev)
    rel = (p - older[:, None])
    sp = torch.where(rel < 0, p, older[:, None] + path.gather(1, rel.clamp(0, path.shape[1] - 1)))
    moves = (p < new[:, None]) & (ok & ~ended)[:, None]
    sp = torch.where(moves, sp, 0)
    src = page_id.gather(1, (sp // page).clamp(0, width - 1)) * page + sp % page
    dst = tables_out.long().clamp(min=0).gather(1, (p // page).clamp(0, width - 1)) * page + p % page
    moves = moves & (src != dst)
    _move(s["pools"], page, src[moves], dst[moves])
    tables.copy_(tables_out)
    i32 = torch.int32
    return dict(lengths=new.to(i32), free=torch.stack([(head + taken) % n_ring, count - taken + given, (~ok).sum()]).to(i32),
                tables=tables, ring=ring, refs=refs, pools=s["pools"])


def _fork(s):
    page, tables, ring, refs = s["case"]["page"], s["tables"], s["ring"], s["refs"]
    dev, n_ring = tables.device, ring.shape[0]
    src, dst = s["src"].long(), s["dst"].long()
    head, count = s["free"][0].long(), s["free"][1].long()
    length = s["lengths"].long()[src]
    full, held = length // page, (length + page - 1) // page
    need = held - full
    upto = need.cumsum(0)
    ok = (need == 0) | (upto <= count)
    fresh = ring[(head + upto - need) % n_ring]
    col = torch.arange(tables.shape[1], device=dev)
    rows = tables[src]
    last = rows.gather(1, full.clamp(max=tables.shape[1] - 1)[:, None])[:, 0]
    shares = (col < full[:, None]) & ok[:, None]
    refs.index_add_(0, rows.long().clamp(min=0).flatten(), shares.flatten().to(torch.int32))
    takes = (col == full[:, None]) & (ok & (need > 0))[:, None]
    tables[dst] = torch.where(shares, rows, torch.where(takes, fresh[:, None], tables[dst]))
    off = torch.arange(page, device=dev)
    moves = (off < (length % page)[:, None]) & ok[:, None]
    _move(s["pools"], page, (last.long()[:, None] * page + off)[moves], (fresh.long()[:, None] * page + off)[moves])
    lengths = s["lengths"].clone()
    lengths[dst] = torch.where(ok, length, 0).to(torch.int32)
    taken = torch.where(ok, need, 0).sum()
    return dict(lengths=lengths, free=torch.stack([(head + taken) % n_ring, count - taken, (~ok).sum()]).to(torch.int32), tables=tables,
                ring=ring, refs=refs, pools=s["pools"])


def work(case):
    op = case["op"]
    if op in ("tree", "attend"):
        r = _requests(case)
        n, rows = len(r), sum(b for _, b, _ in r)
        words = _pages(case["nodes"], 64)
        if op == "tree":
            return {"bytes": 12 * rows + 8 * words * rows + 12 * n + (4 + 8 * words) * case["padding"], "flops": 0}
        heads, kv_heads, dim, page = case["heads"], case["kv_heads"], case["dim"], case["page"]
        live = [(a, b) for a, b, refused in r if b and not refused]
        c_size = 1 if case["cache"] == "e4m3" else 2
        cached = sum(a for a, _ in live)
        # every new token sees the older ones and itself at least; a chain half of the new ones
        pairs = sum(b * (a - b) + (b if case["tree"] else b * (b + 1) // 2) for a, b in live)
        return {"bytes": cached * kv_heads * dim * 2 * c_size + rows * heads * dim * 2 * (3 if case["gate"] else 2)
                + 4 * sum(_pages(a, page) for a, _ in live) + (8 * words * rows if case["tree"] else 0) + 8 * n,
                "flops": 4 * heads * dim * pairs}
    page, row = case["page"], case["kv_heads"] * case["dim"] * (1 if case["cache"] == "e4m3" else 2)
    if op == "keep":
        older, new, kept = _drafts(case)
        moved = 0 if case["chain"] else sum(max(0, k) for k in kept)
        gone = sum(_pages(a + m, page) - (_pages(a + k, page) if k >= 0 else 0) for a, m, k in zip(older, new, kept))
        return {"bytes": 2 * moved * row * case["pools"] + 16 * len(new) + (8 if not case["shared"] else 16) * gone, "flops": 0}
    older = _ratios(case["shortest"], case["longest"], case["sources"])
    taken, moved = 0, 0
    for _ in range(case["copies"]):
        for a in older:
            if a % page == 0:
                continue
            taken += 1
            moved += a % page if taken <= case["spare"] else 0
    return {"bytes": 2 * moved * row * case["pools"] + 16 * case["copies"] * sum(a // page for a in older) + 16 * len(older), "flops": 0}


def exact(case, seed):
    if case["op"] != "attend":
        return None                      # whole numbers, and copies of what is there
    s = prepare(case, seed)
    dim, kv_heads, page = case["dim"], case["kv_heads"], case["page"]
    group = case["heads"] // kv_heads
    out = s["out"].to(torch.float64)
    lengths, starts, slots = s["lengths"].tolist(), s["starts"].tolist(), s["slots"].tolist()
    raw = {n: s[n + "_cache"].view(torch.uint8 if case["cache"] == "e4m3" else torch.int16) for n in "kv"}
    masks = s["masks"].cpu().numpy() if s["masks"] is not None else None
    for b, length in enumerate(lengths):
        lo, hi = starts[b], starts[b + 1]
        if lo == hi or slots[lo] < 0:
            continue
        m = hi - lo
        # the mask over the new tokens, bit by bit
        if masks is None:
            new = torch.ones(m, m, dtype=torch.bool).tril()
        else:
            new = torch.from_numpy(np.unpackbits(masks[lo:hi].view("uint8"), axis=1, bitorder="little")[:, :m].astype(bool))
        hidden = torch.zeros(m, length, dtype=torch.bool)
        hidden[:, length - m:] = ~new
        hidden = hidden.cuda()
        ids = s["tables"][b, : _pages(length, page)].to(torch.int64)
        for h in range(kv_heads):
            k, v = (raw[n][ids, h].view(DTYPES[case["cache"]]).reshape(-1, dim)[:length].to(torch.float64) for n in "kv")
            if s["k_scale"] is not None:
                k, v = k * s["k_scale"][h].to(torch.float64), v * s["v_scale"][h].to(torch.float64)
            mine = slice(h * group, (h + 1) * group)
            score = torch.einsum("igd,jd->gij", s["q"][lo:hi, mine].to(torch.float64), k) / math.sqrt(dim)
            weight = torch.softmax(score.masked_fill(hidden, -math.inf), dim=-1)
            out[lo:hi, mine] = torch.einsum("gij,jd->igd", weight, v)
    if s["gate"] is not None:
        out = out / (1 + torch.exp(-s["gate"].to(torch.float64)))
    return out
