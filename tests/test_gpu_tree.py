"""Tree masks and the attention of several new tokens of a request, on the GPU against the float64 oracle: masks bit for bit,
outputs within bounds derived from their roundings.

Bounds. u(t) is half a step of type t relative to the value. A score is a sum of D products accumulated in fp32, off by at
most D 2^-23 sum|q k| scale =: d; the weight's exponent (the score times log2(e), less the row's base) is rounded to fp32
twice more, off by 2^-22 mag for scores up to mag; so a weight is off by e^(d + 2^-22 mag), by the exponential's own 2^-22
and by its rounding to 16 bits, u(p), and the normaliser likewise but for the rounding. The sum over n tokens adds one fp32
rounding for every 16 of them, and one for each of the times a sum is rescaled or joined (at most n / 64 and 200 of them,
which n / 16 + 232 covers). With S = sum p |v|:
    |err| <= u(out) |out| + S (u(p) + 2 d + 2^-21 mag + (n / 16 + 232) 2^-23) + the smallest step of fp16."""
import numpy as np
import pytest

import oracle.cache_oracle as O
from test_gpu_cache import U, dt, f64, gen_of, ints, randn, torch_
from w4a16_top_mixture_gb300 import build, lib

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    build.build()
    lib.load_library()


# ---------------------------------------------------------------- masks

def random_parents(rng, new, kind):
    out = []
    for n in new:
        for i in range(n):
            out.append(i - 1 if kind == "chain" else -1 if kind == "flat" else int(rng.integers(max(-1, i - 9), i)))
    return out


def u64(t):
    return t.cpu().numpy().view(np.uint64)


@pytest.mark.parametrize("kind", ["random", "chain", "flat"])
@pytest.mark.parametrize("B,most,words,padding", [(1, 1, 1, 0), (1, 64, 1, 3), (3, 65, 2, 0), (40, 17, 4, 5), (7, 256, 4, 70),
                                                  (5, 192, 3, 0), (1000, 9, 1, 1)])
def test_tree_matches_the_oracle(B, most, words, padding, kind):
    torch = torch_()
    rng = np.random.default_rng(B + most)
    new = rng.integers(0, most + 1, B)
    new[-1] = most
    lengths = new + rng.integers(0, 1000, B)
    refused = rng.random(B) < 0.1
    refused[-1] = False
    starts = np.concatenate([[0], np.cumsum(new)])
    rows = int(starts[-1]) + padding
    parents = np.full(rows, 77, np.int32)
    parents[:starts[-1]] = random_parents(rng, new, kind)
    slots = np.full(rows, -1, np.int32)
    for b in range(B):
        if not refused[b]:
            slots[starts[b]:starts[b + 1]] = 5
    c = lib.PagedCache(1, 1, 64, 16, 100, B, 200, max_new=most)
    t = c.tree(ints(parents), ints(starts), ints(lengths), slots=ints(slots), words=words)
    torch.cuda.synchronize()
    masks, positions = O.tree(parents, starts, lengths, refused, rows, words)
    np.testing.assert_array_equal(u64(t.masks), masks)
    np.testing.assert_array_equal(t.positions.cpu().numpy(), positions)
    assert c.status() == (0, 0)
    if words == -(-most // 64):                               # the words that the handle's trees need, unless given
        assert c.tree(ints(parents), ints(starts), ints(lengths)).masks.shape == (rows, words)


def test_tree_reports_parents_and_starts_that_cannot_be():
    c = lib.PagedCache(1, 1, 64, 16, 100, 4, 20, max_new=40)
    ok = ints([-1, 0, 1, 0])
    for bad in ([-1, 1, 1, 0], [0, 0, 1, 0], [-1, 0, 1, -2], [-1, 0, 3, 0], [-1, 0, 2 ** 31 - 1, 0]):
        t = c.tree(ints(bad), ints([0, 4]), ints([9]))
        want = [p if -1 <= p < i else -1 for i, p in enumerate(bad)]
        masks, positions = O.tree(want, [0, 4], [9], [False], 4, 1)
        assert (u64(t.masks) == masks).all() and t.positions.tolist() == positions.tolist()
        assert c.status() == (-1, 16)
    for starts, lengths, flag in (([0, 5], [9], 16), ([-1, 4], [9], 16), ([3, 2], [9], 16), ([0, 4], [3], 2), ([0, 4], [-1], 2),
                                  ([0, 4], [321], 2)):
        t = c.tree(ok, ints(starts), ints(lengths))
        assert c.status()[1] == flag
        assert flag == 16 or (t.masks == 0).all()
    c = lib.PagedCache(1, 1, 64, 16, 100, 4, 20, max_new=3)    # more new tokens than the handle takes
    assert (c.tree(ok, ints([0, 4]), ints([9])).masks == 0).all() and c.status() == (-1, 16)


# ---------------------------------------------------------------- attention

def tree_case(reqs, Hq, Hkv, D, page, act, cache, seed, gate=True, masks="tree", words=1, padding=0, gain=1.0):
    """reqs: (older, new, refused) of each request. NaN past every request's end and in a page of nobody."""
    torch = torch_()
    g, rng = gen_of(seed), np.random.default_rng(seed)
    B = len(reqs)
    new = np.array([n for _, n, _ in reqs])
    lengths = np.array([o + (0 if r else n) for o, n, r in reqs])
    starts = np.concatenate([[0], np.cumsum(new)])
    rows = int(starts[-1]) + padding
    held = -(-lengths // page)
    n_pages, width = int(held.sum()) + 2, int(held.max()) + 1
    order = torch.randperm(n_pages, generator=g, device="cuda").tolist()
    tables = np.full((B, width), 2 ** 30, np.int32)
    at = 0
    for b in range(B):
        tables[b, :held[b]] = order[at:at + held[b]]
        at += held[b]
    pool = randn(g, (n_pages, 2, Hkv, page, D), cache, 8.0 if cache == "e4m3" else 1.0)
    raw = pool.view(torch.uint8) if cache == "e4m3" else pool.view(torch.int16)
    nan = 0x7F if cache == "e4m3" else 0x7FFF
    for b, n in enumerate(lengths.tolist()):
        if n % page:
            raw[tables[b, n // page], :, :, n % page:] = nan
    raw[order[at]] = nan
    x = randn(g, (rows, Hq, 2, D), act, 1.5 * gain)
    slots = np.full(rows, -1, np.int32)
    for b, (_, n, r) in enumerate(reqs):
        slots[starts[b]:starts[b + 1]] = -1 if r else 3
    d = dict(q=x[:, :, 0], starts=ints(starts), tables=ints(tables), lengths=ints(lengths), k_cache=pool[:, 0], v_cache=pool[:, 1],
             slots=ints(slots))
    if gate:
        d["gate"] = x[:, :, 1]
    if masks == "tree":
        m, _ = O.tree(random_parents(rng, new, "random"), starts, lengths, [r for _, _, r in reqs], rows, words)
    elif masks == "any":                                       # no tree: rows that see nothing new, everything, anything
        m = rng.integers(0, 2 ** 63, (rows, words)).astype(np.uint64) * np.uint64(2) + rng.integers(0, 2, (rows, words)).astype(np.uint64)
        m[::3] = 0
        m[1::5] = np.uint64(2 ** 64 - 1)
    if masks:
        d["masks"] = torch.from_numpy(m.view(np.int64)).cuda()
    if cache == "e4m3":
        d["k_scale"] = torch.rand(Hkv, generator=g, device="cuda") * 0.1 + 0.05
        d["v_scale"] = torch.rand(Hkv, generator=g, device="cuda") * 0.1 + 0.05
    return d, n_pages, width


def oracle_of(d, D, scale=None):
    k, v = f64(d["k_cache"]), f64(d["v_cache"])
    if "k_scale" in d:
        k, v = k * f64(d["k_scale"])[:, None, None], v * f64(d["v_scale"])[:, None, None]
    starts, slots = d["starts"].cpu().numpy(), d["slots"].cpu().numpy()
    refused = [starts[b] < starts[b + 1] and slots[starts[b]] < 0 for b in range(len(starts) - 1)]
    return O.attend_tree(f64(d["q"]), starts, refused, u64(d["masks"]) if "masks" in d else None, d["tables"].cpu().numpy(),
                         d["lengths"].cpu().numpy(), k, v, D ** -0.5 if scale is None else scale, f64(d.get("gate")))


def tree_check(d, out, D, act, cache, scale=None, finite=True):
    want, size, mag, seen = oracle_of(d, D, scale)
    rows = int(d["starts"][-1])
    want, size, mag, seen, got = want[:rows], size[:rows], mag[:rows], seen[:rows], f64(out)[:rows]
    up = U["f16"] if cache == "e4m3" else U[act]
    delta = D * 2.0 ** -23 * mag
    tol = U[act] * np.abs(want) + size * (up + 2 * delta + 2.0 ** -21 * mag + (seen / 16 + 232) * 2.0 ** -23) + 2.0 ** -24
    assert not finite or np.isfinite(want).all()
    ok = np.isfinite(want)
    assert (np.isfinite(got) == ok).all(), np.argwhere(np.isfinite(got) != ok)[:4]
    bad = np.abs(np.where(ok, got, 0) - np.where(ok, want, 0)) > np.where(ok, tol, 0)
    assert not bad.any(), (np.argwhere(bad)[:4], np.abs(got - want)[bad][:4], tol[bad][:4])
    assert (got[np.broadcast_to(seen == 0, got.shape)] == 0).all()


def run_tree(reqs, Hq, Hkv, D, page, act, cache, seed, gate=True, masks="tree", words=1, padding=0):
    torch = torch_()
    d, n_pages, width = tree_case(reqs, Hq, Hkv, D, page, act, cache, seed, gate, masks, words, padding)
    most = max(n for _, n, _ in reqs)
    c = lib.PagedCache(Hq, Hkv, D, page, n_pages, len(reqs), width, dtype=act, cache_dtype=cache, max_new=max(1, most))
    out = torch.full_like(d["q"], 7.0).contiguous()
    c.attend_tree(**d, out=out)
    again = c.attend_tree(**d, out=out.clone())
    assert c.status() == (0, 0)
    tree_check(d, out, D, act, cache)
    assert (out[int(d["starts"][-1]):] == 7.0).all()          # rows past the last token, as they were
    assert torch.equal(out, again)                            # sums in a fixed order
    c.close()


EDGES = [(0, 1, 0), (1, 1, 0), (0, 0, 0), (0, 5, 0), (14, 1, 0), (14, 2, 0), (15, 2, 0), (50, 3, 1), (60, 4, 0), (63, 1, 0), (60, 9, 0),
         (3, 0, 0), (127, 1, 0), (121, 16, 0), (0, 16, 0), (255, 7, 0), (1000, 13, 0)]
WIDE = [(0, 64, 0), (1, 63, 0), (77, 64, 0), (0, 1, 0), (500, 33, 1), (190, 2, 0), (333, 61, 0)]
CHUNK = [(0, 256, 0), (256, 256, 0), (100, 255, 0), (0, 129, 0), (31, 1, 0)]
SHAPES = [(16, 2, 256, 16, "f16", "f16", True), (16, 2, 256, 16, "bf16", "e4m3", True), (32, 8, 128, 64, "bf16", "bf16", False),
          (5, 1, 64, 32, "f16", "e4m3", True), (9, 3, 128, 256, "f16", "f16", True), (64, 1, 64, 16, "f16", "f16", False),
          (17, 1, 256, 128, "bf16", "bf16", True), (32, 1, 256, 64, "f16", "e4m3", False), (6, 6, 64, 128, "bf16", "bf16", True),
          (14, 2, 128, 16, "bf16", "e4m3", True), (1, 1, 64, 16, "bf16", "e4m3", False), (8, 8, 128, 16, "f16", "e4m3", True)]


@pytest.mark.parametrize("Hq,Hkv,D,page,act,cache,gate", SHAPES)
@pytest.mark.parametrize("masks", ["tree", None, "any"])
def test_attend_tree_edges(Hq, Hkv, D, page, act, cache, gate, masks):
    run_tree(EDGES, Hq, Hkv, D, page, act, cache, Hq + D + page, gate, masks, 1, 3)


@pytest.mark.parametrize("Hq,Hkv,D,page,act,cache,gate", SHAPES)
def test_attend_tree_wide(Hq, Hkv, D, page, act, cache, gate):
    run_tree(WIDE, Hq, Hkv, D, page, act, cache, Hq + D, gate, "tree", 1)


@pytest.mark.parametrize("Hq,Hkv,D,page,act,cache,gate", [SHAPES[i] for i in (0, 1, 2, 4, 8)])
@pytest.mark.parametrize("masks", [None, "any"])
def test_attend_tree_chunks(Hq, Hkv, D, page, act, cache, gate, masks):
    run_tree(CHUNK, Hq, Hkv, D, page, act, cache, D, gate, masks, 4)


@pytest.mark.parametrize("reqs,shape", [([(20000, 5, 0)], 0), ([(30011, 3, 0)], 1), ([(9000, 17, 0), (0, 0, 0), (1, 1, 0), (5000, 4, 0)], 2),
                                        ([(300 + i, 1 + i % 9, 0) for i in range(200)], 3), ([(700, 6, 0)] * 60, 9), ([(40, 2, 1)] * 3, 0),
                                        ([(0, 0, 0)] * 4 + [(9, 1, 0)], 2), ([(2500, 30, 0), (3000, 64, 0)], 10)],
                         ids=["long", "long8", "ragged", "many", "even", "refused", "empty", "one-head"])
def test_attend_tree_batches(reqs, shape):
    run_tree(reqs, *SHAPES[shape][:6], 7, SHAPES[shape][6], "tree", 1, 2)


@pytest.mark.parametrize("kind", ["keys", "values", "both", "infinite values"])
@pytest.mark.parametrize("Hq,Hkv,D,page,act,cache", [(16, 2, 256, 16, "f16", "f16"), (4, 1, 64, 32, "bf16", "e4m3"), (8, 4, 128, 64, "bf16", "bf16")])
def test_attend_tree_what_a_row_does_not_see_has_no_effect(Hq, Hkv, D, page, act, cache, kind):
    """NaN and infinities in keys and values of new tokens: rows that see them get what the formula gives, others nothing."""
    torch = torch_()
    if cache == "e4m3" and kind == "infinite values":
        pytest.skip("e4m3 has no infinities")
    reqs = [(37, 12, 0), (0, 20, 0), (130, 7, 0)]
    d, n_pages, width = tree_case(reqs, Hq, Hkv, D, page, act, cache, 5, False, "tree", 1)
    starts, tables = d["starts"].tolist(), d["tables"].cpu().numpy()
    for b, (older, n, _) in enumerate(reqs):
        for j in (2, n - 1):                                  # a token with descendants, mostly, and a leaf
            pos = older + j
            at = (int(tables[b, pos // page]), 0, pos % page)
            if kind in ("keys", "both"):
                d["k_cache"][at[0], at[1], at[2], 5] = float("nan")
            if kind in ("values", "both"):
                d["v_cache"][at[0], at[1], at[2], 7] = float("nan")
            if kind == "infinite values":
                d["v_cache"][at[0], at[1], at[2], 7] = float("inf")
                d["v_cache"][at[0], at[1], at[2], 9] = float("-inf")
    c = lib.PagedCache(Hq, Hkv, D, page, n_pages, len(reqs), width, dtype=act, cache_dtype=cache, max_new=20)
    out = c.attend_tree(**d)
    assert c.status() == (0, 0)
    tree_check(d, out, D, act, cache, finite=False)
    want = oracle_of(d, D)[0]
    assert not np.isfinite(want).all() and np.isfinite(want).any(axis=(1, 2)).any()
    inf = np.isinf(want)
    assert (f64(out)[inf] == want[inf]).all()


def test_attend_tree_bad_pages_and_lengths():
    torch = torch_()
    reqs = [(90, 5, 0), (50, 5, 0), (10, 3, 0)]
    for cache in ("f16", "e4m3"):
        d, n_pages, width = tree_case(reqs, 4, 2, 64, 16, "f16", cache, 8)
        c = lib.PagedCache(4, 2, 64, 16, n_pages, 3, width, cache_dtype=cache, max_new=5)
        for bad in (-1, n_pages, 2 ** 31 - 1, -2 ** 31):
            t = d["tables"].clone()
            t[0, 1] = t[1, 3] = bad
            out = c.attend_tree(**{**d, "tables": t})
            assert c.status() == (-1, 4)
            tree_check({**d, "tables": t}, out, 64, "f16", cache)
        good = c.attend_tree(**d)
        for change, flag in ((dict(lengths=[95, 4, 13]), 2), (dict(lengths=[95, -3, 13]), 2), (dict(lengths=[95, width * 16 + 1, 13]), 2),
                             (dict(starts=[0, 5, 4, 13]), 16), (dict(starts=[0, 5, 14, 13]), 16)):
            out = torch.full_like(good, 3.0)
            c.attend_tree(**{**d, **{k: ints(v) for k, v in change.items()}}, out=out)
            assert c.status()[1] & flag
            if change != dict(starts=[0, 5, 4, 13]):          # there the last request's rows overlap the first one's
                assert torch.equal(out[:5], good[:5])
            if flag == 2:
                assert (out[5:10] == 0).all() and torch.equal(out[10:], good[10:])
    c = lib.PagedCache(4, 2, 64, 16, n_pages, 3, width, cache_dtype="e4m3", max_new=4)   # fewer new tokens than the call brings
    out = c.attend_tree(**d)
    assert c.status() == (-1, 16) and (out[:10] == 0).all() and torch.equal(out[10:], good[10:])


def test_attend_tree_in_place_scales_and_streams():
    torch = torch_()
    reqs = [(3000, 9, 0), (0, 4, 0), (700, 12, 0)]
    d, n_pages, width = tree_case(reqs, 8, 2, 128, 16, "f16", "f16", 9, True, "tree", 1)
    c = lib.PagedCache(8, 2, 128, 16, n_pages, 3, width, max_new=12)
    base = c.attend_tree(**d)
    for name in ("q", "gate"):
        x = d[name].clone(memory_format=torch.preserve_format)
        assert torch.equal(c.attend_tree(**{**d, name: x}, out=x), base)
    for scale in (0.0, -0.07, 1e-30, 0.5):
        tree_check(d, c.attend_tree(**d, scale=scale), 128, "f16", "f16", scale)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    out = c.attend_tree(**d, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(out, base)
    # captured, and replayed with other lengths and queries in place
    graph, out = torch.cuda.CUDAGraph(), torch.zeros_like(base)
    with torch.cuda.graph(graph):
        c.attend_tree(**d, out=out)
    d["q"].mul_(0.5)
    d["lengths"].sub_(ints([1000, 0, 3]))
    d["v_cache"].nan_to_num_()
    d["k_cache"].nan_to_num_()
    graph.replay()
    torch.cuda.synchronize()
    tree_check(d, out, 128, "f16", "f16")
    assert c.status() == (0, 0)


def test_attend_tree_long_flat_tails_and_steep_scores():
    """One high score over a long tail of low ones whose sum counts; scores that rise along the sequence, so that the running
    maximum rises at nearly every tile."""
    torch = torch_()
    n, D = 40000, 128
    d, n_pages, width = tree_case([(n, 3, 0), (n // 4, 2, 0)], 4, 1, D, 64, "f16", "f16", 10, False, None)
    q = torch.zeros_like(d["q"])
    q[..., 0] = 1.0
    for shape in ("tail", "rising", "falling"):
        for b, length in enumerate(d["lengths"].tolist()):
            pos = torch.arange(length, device="cuda")
            s = {"tail": torch.where(pos == 17, 0.0, -15.0), "rising": pos * (300.0 / length), "falling": -pos * (300.0 / length)}[shape]
            page, off = d["tables"][b].long()[pos // 64], pos % 64
            d["k_cache"][page, 0, off, 0] = s.half()
            d["v_cache"][page, 0, off, 1] = torch.where(pos == 17, 0.0, 1.0).half()
        dd = {**d, "q": q}
        c = lib.PagedCache(4, 1, D, 64, n_pages, 2, width, max_new=3)
        tree_check(dd, c.attend_tree(**dd, scale=1.0), D, "f16", "f16", 1.0)


def test_a_drafted_step_end_to_end():
    """Plan, tree, write, attention, keep, and the next step, as they are used together: what is kept attends as if it had been
    written alone."""
    torch = torch_()
    rng = np.random.default_rng(12)
    B, Hq, Hkv, D, page, width, n_pages, new = 3, 4, 2, 64, 16, 10, 40, 9
    c = lib.PagedCache(Hq, Hkv, D, page, n_pages, B, width, rope_dim=32, rope_theta=1e4, max_new=new)
    gen = gen_of(13)
    kc, vc = torch.zeros(c.pool_shape, device="cuda").half(), torch.zeros(c.pool_shape, device="cuda").half()
    k2, v2 = kc.clone(), vc.clone()
    pools, pools2 = c.pools([kc, vc]), c.pools([k2, v2])
    rows = B * new

    def fresh():
        return (ints(np.zeros(B)), torch.full((B, width), -1, dtype=torch.int32, device="cuda"),
                torch.arange(n_pages, dtype=torch.int32, device="cuda"), ints([0, n_pages, 0]))
    lengths, tables, ring, state = fresh()
    l2, t2, r2, s2 = fresh()
    for step in range(4):
        x = randn(gen, (rows, Hq + 2 * Hkv, D), "f16")
        q, k, v = x[:, :Hq], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:]
        parents = random_parents(rng, [new] * B, "random")
        p = c.plan(lengths, ints([new] * B), tables, ring, state, rows)
        t = c.tree(ints(parents), p.starts, p.lengths, slots=p.slots)
        qr = c.write(q, k, v, t.positions, p.slots, kc, vc)
        y = c.attend_tree(qr, p.starts, tables, p.lengths, kc, vc, masks=t.masks, slots=p.slots)
        # a path from a random token up to the root
        path, counts = np.zeros((B, new), np.int32), []
        for b in range(B):
            j, up = int(rng.integers(0, new)), []
            while j >= 0:
                up.append(j)
                j = parents[b * new + j]
            counts.append(len(up))
            path[b, :len(up)] = up[::-1]
        kept = c.keep(ints(counts), p.lengths, tables, ring, p.free_state, pools, starts=p.starts, slots=p.slots, path=ints(path))
        lengths, state = kept.lengths, kept.free_state
        # the same tokens as a chain of their own
        rows2 = torch.tensor([b * new + int(j) for b in range(B) for j in path[b, :counts[b]]], device="cuda")
        p2 = c.plan(l2, ints(counts), t2, r2, s2, len(rows2))
        q2 = c.write(q[rows2], k[rows2], v[rows2], p2.positions, p2.slots, k2, v2)
        y2 = c.attend_tree(q2, p2.starts, t2, p2.lengths, k2, v2, slots=p2.slots)
        l2, s2 = p2.lengths, p2.free_state
        assert torch.equal(lengths, l2) and lengths.min() > 0
        err = (y[rows2].float() - y2.float()).abs().max().item()
        assert err <= 2.0 ** -10 * y2.float().abs().max().item() + 2.0 ** -9   # two roundings of weights and outputs of about 1
        for b in range(B):
            for pos in range(int(lengths[b])):
                a, z = (int(tab[b, pos // page]) for tab in (tables, t2))
                assert torch.equal(kc[a, :, pos % page], k2[z, :, pos % page]) and torch.equal(vc[a, :, pos % page], v2[z, :, pos % page])
    # a fork goes on with the same tokens, and gives its shared pages back
    refs = torch.zeros(n_pages, dtype=torch.int32, device="cuda")
    big = lib.PagedCache(Hq, Hkv, D, page, n_pages, B + 2, width, rope_dim=32, rope_theta=1e4, max_new=new)
    more = torch.cat([tables, torch.full((2, width), -1, dtype=torch.int32, device="cuda")])
    at = big.pools([kc, vc])
    f = big.fork(ints([0, 1]), ints([3, 4]), torch.cat([lengths, ints([0, 0])]), more, ring, state, refs, at)
    q1 = randn(gen, (B + 2, Hq, D), "f16")
    q1[3:] = q1[:2]
    a1 = big.attend(q1, more, f.lengths, kc, vc)
    assert torch.equal(a1[3:], a1[:2])
    free = int(state[1])
    done = big.keep(ints([-1, -1, int(lengths[2]), -1, -1]), f.lengths, more, ring, f.free_state, at, refs=refs)
    held = -(-int(lengths[2]) // page)
    assert int(done.free_state[1]) == n_pages - held > free and (refs == 0).all() and c.status() == (0, 0) and big.status() == (0, 0)
    back = [int(ring[(int(done.free_state[0]) + i) % n_pages]) for i in range(n_pages - held)]
    assert len(set(back)) == n_pages - held
