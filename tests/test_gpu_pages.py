"""Keeping a path of a step's new tokens and forking requests, on the GPU against the oracle: whole numbers and copies, so
every output is compared bit for bit."""
import numpy as np
import pytest

import oracle.cache_oracle as O
from test_gpu_cache import dt, gen_of, ints, torch_
from w4a16_top_mixture_gb300 import build, lib

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    build.build()
    lib.load_library()


def pool_bits(torch, shape, name, gen):
    """A pool of random bits (a copy keeps every bit, those of NaN too)."""
    if name == "e4m3":
        return torch.randint(0, 256, shape, generator=gen, device="cuda", dtype=torch.uint8).view(dt(name))
    return torch.randint(-2 ** 15, 2 ** 15, shape, generator=gen, device="cuda", dtype=torch.int16).view(dt(name))


def bits(t):
    torch = torch_()
    return t.view(torch.uint8 if t.element_size() == 1 else torch.int16).cpu().numpy()


def tables_for(rng, lengths, page, spare, shared=()):
    """Tables and a ring for the lengths; shared: (a, b, pages): b's first pages are a's. Returns tables, ring, state, refs."""
    held = -(-np.asarray(lengths) // page)
    n_pages = int(held.sum()) + spare
    order = rng.permutation(n_pages).astype(np.int32)
    tables = np.full((len(lengths), int(held.max()) + 1), -5, np.int32)
    at = 0
    for b, h in enumerate(held):
        tables[b, :h] = order[at:at + h]
        at += h
    free, refs = list(order[at:]), np.zeros(n_pages, np.int32)
    for a, b, n in shared:
        free += list(tables[b, :n])
        tables[b, :n] = tables[a, :n]
        refs[tables[a, :n]] += 1
    head = int(rng.integers(0, n_pages))
    ring = np.full(n_pages, -9, np.int32)
    ring[(head + np.arange(len(free))) % n_pages] = free
    return tables, ring, np.array([head, len(free), 0], np.int32), refs, n_pages


def run_keep(c, pools, counts, lengths, tables, ring, state, starts=None, slots=None, path=None, refs=None, in_place=False):
    torch = torch_()
    ln, fs, tb, rg = ints(lengths), ints(state), ints(tables), ints(ring)
    rf = ints(refs) if refs is not None else None
    r = c.keep(ints(counts), ln, tb, rg, fs, pools, starts=ints(starts) if starts is not None else None,
               slots=ints(slots) if slots is not None else None, path=ints(path) if path is not None else None, refs=rf,
               out=lib.CacheState(ln, fs) if in_place else None)
    torch.cuda.synchronize()
    return [t.cpu().numpy() if t is not None else None for t in (r.lengths, r.free_state, tb, rg, rf)]


NAMES = ("lengths", "state", "tables", "ring", "refs")


def compare(got, want):
    for name, g, w in zip(NAMES, got, want):
        if w is not None:
            np.testing.assert_array_equal(g, w, err_msg=name)


def paths(rng, new, counts, width):
    p = np.full((len(new), width), -3, np.int32)
    for b, (n, k) in enumerate(zip(new, counts)):
        if k > 0:
            p[b, :k] = np.sort(rng.choice(n, k, replace=False))
    return p


# requests, page, longest older, most new, share of ended ones, pairs that share, spare pages
KEEPS = [(1, 16, 40, 1, 0.0, 0, 2), (1, 16, 0, 7, 0.0, 0, 1), (5, 32, 90, 17, 0.3, 2, 3), (16, 16, 200, 64, 0.2, 5, 40),
         (17, 64, 500, 256, 0.1, 8, 2), (129, 16, 100, 33, 0.3, 60, 4), (300, 128, 700, 20, 0.5, 100, 0), (4096, 16, 20, 5, 0.2, 2000, 90)]


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("cache,heads,dim", [("f16", 2, 64), ("e4m3", 1, 64), ("bf16", 3, 256), ("e4m3", 2, 256)])
@pytest.mark.parametrize("B,page,longest,most,p_end,pairs,spare", KEEPS)
def test_keep_matches_the_oracle(B, page, longest, most, p_end, pairs, spare, cache, heads, dim, in_place):
    if B > 300 and dim > 64:
        pytest.skip("a pool of this many requests is tried with small rows alone")
    torch = torch_()
    rng = np.random.default_rng(B + page + dim)
    older, new = rng.integers(0, longest + 1, B), rng.integers(0, most + 1, B)
    lengths = older + new
    starts = np.concatenate([[0], np.cumsum(new)])
    # pairs share pages up to the whole of their common reach, so that tokens move into shared pages and end in them
    shared = [(2 * i, 2 * i + 1, int(rng.integers(0, min(-(-lengths[2 * i] // page), -(-lengths[2 * i + 1] // page)) + 1)))
              for i in range(pairs)]
    tables, ring, state, refs, n_pages = tables_for(rng, lengths, page, spare, shared)
    c = lib.PagedCache(heads, heads, dim, page, n_pages, B, tables.shape[1], dtype="bf16" if cache == "bf16" else "f16",
                       cache_dtype=cache, max_new=max(1, most))
    gen = gen_of(B)
    pools = [pool_bits(torch, (n_pages, heads, page, dim), cache, gen) for _ in range(3)]
    at = c.pools(pools)
    counts = np.minimum(new, rng.integers(0, most + 1, B))
    counts = np.where(rng.random(B) < p_end, -1 - rng.integers(0, 2, B), counts)
    for path in (None, paths(rng, new, counts, max(1, int(counts.max())))):
        # without refs shared pages would be written by both: the pairs only where refs count
        for rf in ((refs,) if pairs else (None, refs)):
            before = [bits(p).copy() for p in pools]
            want = O.keep(counts, lengths, starts, np.zeros(B, bool), path, tables, ring, state, rf, before, page, n_pages)
            got = run_keep(c, at, counts, lengths, tables, ring, state, starts, None, path, rf, in_place)
            compare(got, want)
            for p, w in zip(pools, want[5]):
                np.testing.assert_array_equal(bits(p), w)
            assert c.status() == (0, 0)
    c.close()


def test_keep_goes_back_to_lengths_without_starts():
    torch = torch_()
    rng = np.random.default_rng(3)
    lengths, counts = np.array([100, 0, 33, 64, 20000]), np.array([17, 0, -1, 64, 160])
    tables, ring, state, refs, n_pages = tables_for(rng, lengths, 16, 9, [(0, 3, 4)])
    c = lib.PagedCache(1, 1, 64, 16, n_pages, 5, tables.shape[1], max_new=1)
    pools = [pool_bits(torch, (n_pages, 1, 16, 64), "f16", gen_of(1))]
    at = c.pools(pools)
    for rf in (None, refs):
        before = [bits(p).copy() for p in pools]
        want = O.keep(counts, lengths, None, None, None, tables, ring, state, rf, before, 16, n_pages)
        compare(run_keep(c, at, counts, lengths, tables, ring, state, refs=rf), want)
        np.testing.assert_array_equal(bits(pools[0]), want[5][0])
    assert c.status() == (0, 0)


def test_keep_leaves_refused_requests_as_they_were():
    torch = torch_()
    rng = np.random.default_rng(4)
    lengths, new = np.array([40, 30, 10]), np.array([8, 5, 3])        # the plan refused the second: 30 older tokens
    starts = np.concatenate([[0], np.cumsum(new)])
    slots = np.zeros(16, np.int32)
    slots[8:13] = -1
    tables, ring, state, _, n_pages = tables_for(rng, lengths, 16, 4)
    c = lib.PagedCache(1, 1, 64, 16, n_pages, 3, tables.shape[1], max_new=8)
    pools = [pool_bits(torch, (n_pages, 1, 16, 64), "f16", gen_of(1))]
    counts, path = np.array([2, 0, 1]), np.array([[3, 7], [0, 0], [2, 0]])
    want = O.keep(counts, lengths, starts, [False, True, False], path, tables, ring, state, None, [bits(pools[0])], 16, n_pages)
    got = run_keep(c, c.pools(pools), counts, lengths, tables, ring, state, starts, slots, path)
    compare(got, want)
    np.testing.assert_array_equal(bits(pools[0]), want[5][0])
    assert list(got[0]) == [34, 30, 8] and c.status() == (0, 0)


BAD = [dict(counts=[9, 1]), dict(path=[[3, 3], [0, 0]]), dict(path=[[4, 2], [0, 0]]), dict(path=[[1, 8], [0, 0]]),
       dict(path=[[-1, 2], [0, 0]]), dict(starts=[0, -1, 5]), dict(starts=[0, 9, 5]), dict(starts=[-2, 8, 13]),
       dict(starts=[0, 60, 61]), dict(lengths=[-1, 30]), dict(lengths=[1 << 20, 30])]


@pytest.mark.parametrize("change", BAD, ids=str)
def test_keep_reports_what_cannot_be_and_leaves_it(change):
    torch = torch_()
    rng = np.random.default_rng(5)
    base = dict(counts=[2, 1], lengths=[40, 30], starts=[0, 8, 13], path=[[3, 7], [0, 0]])
    tables, ring, state, refs, n_pages = tables_for(rng, [40, 30], 16, 4)
    c = lib.PagedCache(1, 1, 64, 16, n_pages, 2, tables.shape[1], max_new=8)
    pools = [pool_bits(torch, (n_pages, 1, 16, 64), "f16", gen_of(1))]
    before = bits(pools[0]).copy()
    a = {**base, **change}
    got = run_keep(c, c.pools(pools), a["counts"], a["lengths"], tables, ring, state, a["starts"], np.zeros(13, np.int32), a["path"], refs)
    assert got[0][0] == a["lengths"][0]
    assert got[2][0].tolist() == tables[0].tolist()
    used = bits(pools[0])[tables[0, :3]]
    np.testing.assert_array_equal(used, before[tables[0, :3]])
    status, flags = c.status()
    assert status == -1 and flags & (2 if "lengths" in change else 16)
    assert c.status() == (0, 0)


def test_keep_reports_a_count_above_the_paths_places():
    """What lies behind a request's path is not read: another request's path, or nothing that is the call's."""
    torch = torch_()
    rng = np.random.default_rng(8)
    lengths, starts = np.array([40, 30, 50]), np.array([0, 8, 13, 21])
    tables, ring, state, refs, n_pages = tables_for(rng, lengths, 16, 4)
    c = lib.PagedCache(1, 1, 64, 16, n_pages, 3, tables.shape[1], max_new=8)
    pools = [pool_bits(torch, (n_pages, 1, 16, 64), "f16", gen_of(3))]
    before = bits(pools[0]).copy()
    counts, path = np.array([3, 2, 5]), np.array([[0, 1], [2, 3], [4, 5]])
    got = run_keep(c, c.pools(pools), counts, lengths, tables, ring, state, starts, np.zeros(21, np.int32), path, refs)
    assert list(got[0]) == [40, 27, 50]
    assert got[2][[0, 2]].tolist() == tables[[0, 2]].tolist()
    for b in (0, 2):
        used = tables[b, :-(-lengths[b] // 16)]
        np.testing.assert_array_equal(bits(pools[0])[used], before[used])
    assert c.status() == (-1, 16)


def test_keep_page_ids_outside_the_pool_and_a_full_ring():
    torch = torch_()
    rng = np.random.default_rng(6)
    lengths = np.array([64, 64])
    tables, ring, state, refs, n_pages = tables_for(rng, lengths, 16, 3)
    c = lib.PagedCache(1, 1, 64, 16, n_pages, 2, tables.shape[1], max_new=8)
    pools = [pool_bits(torch, (n_pages, 1, 16, 64), "f16", gen_of(1))]
    for bad in (-1, n_pages, -2 ** 31, 2 ** 31 - 1):
        for rf in (None, refs):
            t = tables.copy()
            t[0, 2] = t[1, 3] = bad
            got = run_keep(c, c.pools(pools), [-1, 5], lengths, t, ring, state, [0, 8, 16], None, None, rf)
            assert got[0].tolist() == [0, 61] and c.status() == (-1, 4)
            assert got[1][1] == 3 + 3
    # pages past the ring's room are left out: the state says that all but one are free already
    full = np.array([0, n_pages - 1, 0], np.int32)
    got = run_keep(c, c.pools(pools), [-1, 8], lengths, tables, ring, full, [0, 8, 16])
    want = ring.copy()
    want[n_pages - 1] = tables[0, 0]
    np.testing.assert_array_equal(got[3], want)
    assert got[1].tolist() == [0, n_pages, 0] and c.status() == (-1, 8)
    got = run_keep(c, c.pools(pools), [-1, 8], lengths, tables, ring, np.array([n_pages, 2, 0], np.int32), [0, 8, 16])
    assert c.status()[1] & 8


def test_keep_page_given_back_by_many_goes_to_the_ring_once():
    """300 requests over one prompt end in one call, in any order of the atomics."""
    torch = torch_()
    rng = np.random.default_rng(7)
    B = 300
    lengths = rng.integers(160, 300, B)
    tables, ring, state, refs, n_pages = tables_for(rng, lengths, 16, 5, [(0, b, 10) for b in range(1, B)])
    c = lib.PagedCache(1, 1, 64, 16, n_pages, B, tables.shape[1], max_new=1)
    pools = [pool_bits(torch, (n_pages, 1, 16, 64), "f16", gen_of(1))]
    at = c.pools(pools)
    for alive in (0, 1):                                     # the last one may go on: then its pages stay
        counts = np.full(B, -1)
        counts[B - 1] = lengths[B - 1] if alive else -1
        want = O.keep(counts, lengths, None, None, None, tables, ring, state, refs, [], 16, n_pages)
        for _ in range(5):
            compare(run_keep(c, at, counts, lengths, tables, ring, state, refs=refs), want)
    assert c.status() == (0, 0)


FORKS = [(1, 1, 16, 40, 3), (1, 3, 16, 48, 0), (2, 3, 32, 200, 9), (20, 5, 64, 900, 30), (33, 2, 16, 100, 200), (800, 4, 128, 300, 1000)]


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("cache,heads,dim", [("f16", 2, 64), ("e4m3", 1, 64), ("bf16", 3, 128)])
@pytest.mark.parametrize("sources,copies,page,longest,spare", FORKS)
def test_fork_matches_the_oracle(sources, copies, page, longest, spare, cache, heads, dim, in_place):
    if sources > 100 and heads > 1:
        pytest.skip("a pool of this many requests is tried with small rows alone")
    torch = torch_()
    rng = np.random.default_rng(sources + page)
    B = sources * (1 + copies) + 2
    order = rng.permutation(B)
    lengths = np.zeros(B, np.int64)
    lengths[order[:sources]] = rng.integers(0, longest + 1, sources)
    lengths[order[0]] = longest // page * page                    # whole pages alone
    tables, ring, state, refs, n_pages = tables_for(rng, lengths, page, spare)
    refs[:] = rng.integers(0, 3, n_pages)
    src, dst = np.tile(order[:sources], copies), order[sources:sources * (1 + copies)]
    src = np.where(rng.random(len(src)) < 0.1, -1 - rng.integers(0, 3, len(src)), src)
    c = lib.PagedCache(heads, heads, dim, page, n_pages, B, tables.shape[1], dtype="bf16" if cache == "bf16" else "f16",
                       cache_dtype=cache, max_new=1)
    gen = gen_of(B)
    pools = [pool_bits(torch, (n_pages, heads, page, dim), cache, gen) for _ in range(3)]
    want = O.fork(src, dst, lengths, tables, ring, state, refs, [bits(p) for p in pools], page, n_pages)
    ln, fs, tb, rg, rf = ints(lengths), ints(state), ints(tables), ints(ring), ints(refs)
    r = c.fork(ints(src), ints(dst), ln, tb, rg, fs, rf, c.pools(pools), out=lib.CacheState(ln, fs) if in_place else None)
    torch.cuda.synchronize()
    compare([t.cpu().numpy() for t in (r.lengths, r.free_state, tb, rg, rf)], want)
    for p, w in zip(pools, want[5]):
        np.testing.assert_array_equal(bits(p), w)
    assert c.status() == (0, 0)
    c.close()


def test_fork_leaves_out_entries_that_cannot_be():
    torch = torch_()
    rng = np.random.default_rng(9)
    lengths = np.array([40, 0, 25, 0, 0])
    tables, ring, state, refs, n_pages = tables_for(rng, lengths, 16, 6)
    c = lib.PagedCache(1, 1, 64, 16, n_pages, 16, tables.shape[1], max_new=1)
    pools = [pool_bits(torch, (n_pages, 1, 16, 64), "f16", gen_of(1))]
    # a dst with tokens, one twice, requests out of range, a source that is another entry's dst (empty at the start)
    src, dst = np.array([0, 0, 2, 5, 0, 2, 1, 0]), np.array([2, 1, 1, 3, -1, 9, 4, 3])
    want = O.fork(src, dst, lengths, tables, ring, state, refs, [bits(pools[0])], 16, n_pages)
    ln, fs, tb, rg, rf = ints(lengths), ints(state), ints(tables), ints(ring), ints(refs)
    r = c.fork(ints(src), ints(dst), ln, tb, rg, fs, rf, c.pools(pools))
    torch.cuda.synchronize()
    compare([t.cpu().numpy() for t in (r.lengths, r.free_state, tb, rg, rf)], want)
    assert r.lengths.tolist() == [40, 40, 25, 40, 0] and c.status() == (-1, 16)


def test_calls_without_pools_or_requests():
    torch = torch_()
    c = lib.PagedCache(1, 1, 64, 16, 8, 4, 2, max_new=1)
    none, ring, state = torch.zeros(0, dtype=torch.int32, device="cuda"), torch.arange(8, dtype=torch.int32, device="cuda"), ints([3, 4, 9])
    tables = torch.zeros(0, 2, dtype=torch.int32, device="cuda")
    r = c.keep(none, none, tables, ring, state, c.pools([]))
    assert r.free_state.tolist() == [3, 4, 0]
    r = c.fork(none, none, none, tables, ring, state, torch.zeros(8, dtype=torch.int32, device="cuda"), c.pools([]))
    assert r.free_state.tolist() == [3, 4, 0] and c.status() == (0, 0)
    t = c.tree(none, ints([0]), none)
    assert t.masks.shape == (0, 1)


def test_many_pools_with_page_strides():
    """130 pools, in several launches; keys and values of a layer as views of one tensor."""
    torch = torch_()
    rng = np.random.default_rng(11)
    lengths, new = np.array([50, 3]), np.array([20, 3])
    starts = np.concatenate([[0], np.cumsum(new)])
    tables, ring, state, _, n_pages = tables_for(rng, lengths, 16, 3)
    c = lib.PagedCache(2, 2, 64, 16, n_pages, 2, tables.shape[1], max_new=20)
    gen = gen_of(5)
    both = [pool_bits(torch, (n_pages, 2, 2, 16, 64), "f16", gen) for _ in range(65)]
    pools = [b[:, i] for b in both for i in range(2)]
    counts, path = np.array([3, 1]), np.array([[2, 9, 19], [2, 0, 0]])
    want = O.keep(counts, lengths, starts, [False] * 2, path, tables, ring, state, None, [bits(p.contiguous()) for p in pools], 16, n_pages)
    compare(run_keep(c, c.pools(pools), counts, lengths, tables, ring, state, starts, None, path), want)
    for p, w in zip(pools, want[5]):
        np.testing.assert_array_equal(bits(p.contiguous()), w)


def test_keep_and_fork_replayed_from_a_graph_and_on_another_stream():
    """A step's keep and the forks after it, in place: eager, on another stream, and from a graph with other counts and paths
    in the same tensors."""
    torch = torch_()
    rng = np.random.default_rng(12)
    B, page = 40, 16
    new = rng.integers(1, 20, B)
    lengths = rng.integers(0, 200, B) + new
    starts = np.concatenate([[0], np.cumsum(new)])
    tables, ring, state, refs, n_pages = tables_for(rng, lengths, page, 200, [(0, 1, 1), (2, 3, 1)])
    wide = np.full((B, 20), -5, np.int32)
    wide[:, :tables.shape[1]] = tables
    c = lib.PagedCache(2, 2, 64, page, n_pages, B, 20, max_new=20)
    first = [pool_bits(torch, (n_pages, 2, page, 64), "f16", gen_of(4)) for _ in range(3)]
    start = [ints(x) for x in (lengths, state, wide, ring, refs)]
    counts, path = ints(np.zeros(B)), ints(np.zeros((B, 20)))
    src, dst, st = ints([0, 2, 2]), ints([5, 7, 6]), ints(starts)

    def choose():
        k = np.minimum(new, rng.integers(0, 20, B))
        k[[5, 6, 7]] = -1
        counts.copy_(ints(k))
        path.copy_(ints(paths(rng, new, k, 20)))

    now, pools = [x.clone() for x in start], [p.clone() for p in first]
    at = c.pools(pools)

    def step(stream=None):
        ln, fs, tb, rg, rf = now
        both = lib.CacheState(ln, fs)
        c.keep(counts, ln, tb, rg, fs, at, starts=st, path=path, refs=rf, out=both, stream=stream)
        c.fork(src, dst, ln, tb, rg, fs, rf, at, out=both, stream=stream)

    def run(f):
        for a, b in zip(now + pools, start + first):
            a.copy_(b)
        torch.cuda.synchronize()
        f()
        torch.cuda.synchronize()
        return [x.cpu().numpy() for x in now] + [bits(p).copy() for p in pools]

    choose()
    k = counts.cpu().numpy()
    kept = O.keep(k, lengths, starts, [False] * B, path.cpu().numpy(), wide, ring, state, refs, [bits(p) for p in first], page, n_pages)
    want = O.fork(src.cpu().numpy(), dst.cpu().numpy(), kept[0], kept[2], kept[3], kept[1], kept[4], kept[5], page, n_pages)
    got = run(step)
    compare(got[:5], want)
    for p, w in zip(got[5:], want[5]):
        np.testing.assert_array_equal(p, w)
    side = torch.cuda.Stream()
    for a, b in zip(run(lambda: step(side)), got):
        np.testing.assert_array_equal(a, b)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for _ in range(4):
        choose()
        for a, b in zip(run(graph.replay), run(step)):
            np.testing.assert_array_equal(a, b)
    assert c.status() == (0, 0)


@pytest.mark.parametrize("cache,heads,dim", [("f16", 2, 64), ("e4m3", 1, 128), ("bf16", 1, 256)])
@pytest.mark.parametrize("share", [False, True])
def test_keep_of_256_new_tokens_in_pages_of_16(cache, heads, dim, share):
    """They lie in 17 pages, the most that a request's rows can move over; where two requests share them, all 17 are exchanged."""
    torch = torch_()
    rng = np.random.default_rng(17)
    lengths, new = np.array([271, 271, 300]), np.array([256, 256, 256])
    starts = np.concatenate([[0], np.cumsum(new)])
    tables, ring, state, refs, n_pages = tables_for(rng, lengths, 16, 40, [(0, 1, 17)] if share else [])
    c = lib.PagedCache(heads, heads, dim, 16, n_pages, 3, tables.shape[1], dtype="bf16" if cache == "bf16" else "f16", cache_dtype=cache,
                       max_new=256)
    pools = [pool_bits(torch, (n_pages, heads, 16, dim), cache, gen_of(i)) for i in range(3)]
    path = np.full((3, 256), -3, np.int32)
    path[0, :255], path[1, :128], path[2, :256] = np.arange(1, 256), np.arange(1, 256, 2), np.arange(256)
    counts, before = np.array([255, 128, 256]), [bits(p).copy() for p in pools]
    want = O.keep(counts, lengths, starts, [False] * 3, path, tables, ring, state, refs, before, 16, n_pages)
    compare(run_keep(c, c.pools(pools), counts, lengths, tables, ring, state, starts, None, path, refs), want)
    for p, w in zip(pools, want[5]):
        np.testing.assert_array_equal(bits(p), w)
    assert c.status() == (0, 0) and (not share or (want[2][:2] != tables[:2])[:, :9].all())


@pytest.mark.parametrize("cache", ["f16", "e4m3"])
def test_pages_that_lie_past_2_to_the_32_bytes(cache):
    """Pools whose pages are far apart give what dense ones do: attention with values that are not finite, a path kept, a fork."""
    torch = torch_()
    rng = np.random.default_rng(21)
    n_pages, apart = 90, 1 << 26 if cache == "e4m3" else 1 << 25
    lengths, starts = np.array([70, 30, 0]), np.array([0, 20, 25, 25])
    c = lib.PagedCache(4, 1, 64, 16, n_pages, 3, 6, cache_dtype=cache, max_new=20)
    tables = np.full((3, 6), -1, np.int32)
    tables[0, :5], tables[1, :2] = [89, 88, 3, 80, 77], [85, 86]
    free = [87, 84, 83, 70, 1]
    ring = np.full(n_pages, -9, np.int32)
    ring[:5] = free
    refs = np.zeros(n_pages, np.int32)
    refs[88] = 1                                              # someone else holds it too
    dense = [torch.randn((n_pages, 1, 16, 64), device="cuda", generator=gen_of(i)).to(dt(cache)) for i in range(2)]
    dense[1][80, 0, 3, 9] = float("nan")                      # a new token's value
    far = [torch.empty((n_pages, apart), dtype=dense[0].dtype, device="cuda")[:, :1024].view(n_pages, 1, 16, 64) for _ in dense]
    for a, b in zip(far, dense):
        a.copy_(b)
    q = torch.randn(25, 4, 64, device="cuda", generator=gen_of(5)).half()
    scales = dict(k_scale=torch.ones(1, device="cuda"), v_scale=torch.ones(1, device="cuda")) if cache == "e4m3" else {}
    one, two = (c.attend_tree(q, ints(starts), ints(tables), ints(lengths), *p, **scales) for p in (dense, far))
    assert torch.equal(one.view(torch.int16), two.view(torch.int16)) and one.isnan().any() and not one.isnan().all()
    counts, path = np.array([9, 3, 0]), np.zeros((3, 20), np.int32)
    path[0, :9], path[1, :3] = [0, 2, 3, 5, 7, 11, 13, 17, 19], [0, 2, 4]
    both = []
    for pools in (dense, far):
        at = c.pools(pools)
        ln, fs, tb, rg, rf = ints(lengths), ints([0, 5, 0]), ints(tables), ints(ring), ints(refs)
        s = lib.CacheState(ln, fs)
        c.keep(ints(counts), ln, tb, rg, fs, at, starts=ints(starts), path=ints(path), refs=rf, out=s)
        c.fork(ints([0]), ints([2]), ln, tb, rg, fs, rf, at, out=s)
        both.append([x.tolist() for x in (ln, fs, tb, rg, rf)] + [bits(p[sorted(set(tables[tables >= 0].tolist() + free))].contiguous()) for p in pools])
    want = O.keep(counts, lengths, starts, [False] * 3, path, tables, ring, np.array([0, 5, 0]), refs, [], 16, n_pages)
    want = O.fork([0], [2], want[0], want[2], want[3], want[1], want[4], [], 16, n_pages)
    assert both[0][:5] == [np.asarray(w).tolist() for w in want[:5]] and both[1][:5] == both[0][:5]
    for a, b in zip(both[0][5:], both[1][5:]):
        np.testing.assert_array_equal(a, b)
    assert c.status() == (0, 0)
