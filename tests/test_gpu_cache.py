"""The paged key-value cache's operators on the GPU against the float64 oracle: the page plan bit for bit, the write and
the attention within bounds derived from their roundings.

Bounds. u(t) is half a step of type t relative to the value. Write: y = x * r * g holds a few fp32 roundings and the
rotation a sum of two products with angles good to 2^-21: u(out) |y| + 2^-20 (|a| + |b|). Attention: a score is a sum of D
products accumulated in fp32, off by at most D 2^-23 sum|q k| scale =: d, so a weight is off by e^d and by its rounding to
16 bits, u(p), and the normaliser by e^d; the sum over n tokens adds one fp32 rounding for every 16 of them. With
S = sum p |v|: |err| <= u(out) |out| + S (u(p) + 2 d + (n / 16 + 32) 2^-23), and the smallest step of fp16."""
import numpy as np
import pytest

import oracle.cache_oracle as O
from w4a16_top_mixture_gb300 import build, lib

pytestmark = pytest.mark.gpu

U = {"f16": 2.0 ** -11, "bf16": 2.0 ** -8}


@pytest.fixture(scope="module", autouse=True)
def _lib():
    build.build()
    lib.load_library()


def torch_():
    import torch
    return torch


def dt(name):
    torch = torch_()
    return {"f16": torch.float16, "bf16": torch.bfloat16, "e4m3": torch.float8_e4m3fn}[name]


def randn(gen, shape, name, gain=1.0):
    torch = torch_()
    x = torch.randn(shape, generator=gen, device="cuda") * gain
    return x.clamp(-448, 448).to(dt(name)) if name == "e4m3" else x.to(dt(name))


def f64(t):
    return t.cpu().double().numpy() if t is not None else None


def gen_of(seed):
    torch = torch_()
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def ints(a):
    torch = torch_()
    return torch.as_tensor(np.asarray(a, np.int32), device="cuda")


# ---------------------------------------------------------------- plan

def plan_case(rng, B, page, longest, p_new, p_end, spare, extra_rows, tight_width=False):
    lengths = rng.integers(0, longest + 1, B)
    new = np.where(rng.random(B) < p_new, rng.integers(0, 3 * page, B), 1)
    new = np.where(rng.random(B) < p_end, -1 - rng.integers(0, 3, B), new)
    held = -(-lengths // page)
    n_pages = int(held.sum()) + spare
    width = int((-(-(lengths + np.maximum(new, 0)) // page)).max())
    width = max(1, width - (1 if tight_width else 0), int(held.max()))
    order = rng.permutation(n_pages).astype(np.int32)
    tables = np.full((B, width), -7, np.int32)
    at = 0
    for b in range(B):
        tables[b, :held[b]] = order[at:at + held[b]]
        at += held[b]
    head = int(rng.integers(0, n_pages))
    ring = np.full(n_pages, -9, np.int32)
    ring[(head + np.arange(spare)) % n_pages] = order[at:]
    rows = max(0, int(np.maximum(new, 0).sum()) + extra_rows)
    return lengths.astype(np.int32), new.astype(np.int32), tables, ring, np.array([head, spare, 0], np.int32), rows, n_pages, width


def run_plan(c, lengths, new, tables, ring, state, rows, in_place=False):
    torch = torch_()
    ln, fs, tb, rg = ints(lengths), ints(state), ints(tables), ints(ring)
    out = None
    if in_place:
        e = lambda n: torch.empty(n, dtype=torch.int32, device="cuda")  # noqa: E731
        out = lib.CachePlan(e(rows), e(rows), e(len(lengths) + 1), ln, fs)
    p = c.plan(ln, ints(new) if new is not None else None, tb, rg, fs, rows, out=out)
    torch.cuda.synchronize()
    return [t.cpu().numpy() for t in (*p, tb, rg)]


PLANS = [(1, 16, 40, 0.0, 0.0, 1, 0), (1, 16, 0, 1.0, 0.0, 3, 5), (7, 16, 100, 0.3, 0.2, 20, 3), (33, 32, 500, 0.5, 0.1, 9, 0),
         (127, 64, 900, 0.2, 0.3, 40, 11), (128, 128, 300, 0.1, 0.0, 0, 1), (129, 256, 5000, 0.9, 0.05, 60, 0),
         (1000, 16, 300, 0.3, 0.1, 500, -400), (1025, 16, 33, 0.1, 0.5, 4000, 77), (4096, 32, 90, 0.5, 0.2, 2500, 9)]


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("B,page,longest,p_new,p_end,spare,extra", PLANS)
def test_plan_matches_the_oracle(B, page, longest, p_new, p_end, spare, extra, in_place):
    rng = np.random.default_rng(B + page)
    for tight in (False, True):
        lengths, new, tables, ring, state, rows, n_pages, width = plan_case(rng, B, page, longest, p_new, p_end, spare, extra, tight)
        c = lib.PagedCache(1, 1, 64, page, n_pages, B, width)
        got = run_plan(c, lengths, new, tables, ring, state, rows, in_place)
        want = O.plan(lengths, new, tables, ring, state, rows, page, n_pages)
        for name, g, w in zip(("slots", "positions", "starts", "lengths", "state", "tables", "ring"), got, want):
            np.testing.assert_array_equal(g, w, err_msg=name)
        assert c.status() == (0, 0)
        c.close()


def test_plan_without_new_tokens_gives_each_request_one():
    rng = np.random.default_rng(5)
    lengths, _, tables, ring, state, _, n_pages, width = plan_case(rng, 40, 16, 200, 0, 0, 30, 0)
    c = lib.PagedCache(1, 1, 64, 16, n_pages, 64, width)
    got = run_plan(c, lengths, None, tables, ring, state, 40)
    for g, w in zip(got, O.plan(lengths, None, tables, ring, state, 40, 16, n_pages)):
        np.testing.assert_array_equal(g, w)


def test_plan_of_nothing():
    c = lib.PagedCache(1, 1, 64, 16, 8, 4, 2)
    got = run_plan(c, np.zeros(0), np.zeros(0), np.zeros((0, 2)), np.arange(8), [3, 5, 9], 3)
    assert list(got[0]) == [-1] * 3 and list(got[1]) == [0] * 3 and list(got[2]) == [0] and list(got[4]) == [3, 5, 0]


def test_plan_reports_what_it_cannot_use():
    c = lib.PagedCache(1, 1, 64, 16, 8, 4, 2)
    tables = np.array([[0, 1], [2, 3], [99, -1], [4, -1]])
    got = run_plan(c, [-1, 33, 3, 3], [1, 1, 1, 1], tables, np.arange(8), [0, 0, 0], 4)
    assert list(got[0]) == [-1, -1, -1, 4 * 16 + 3] and list(got[3]) == [-1, 33, 4, 4] and list(got[4]) == [0, 0, 2]
    assert c.status() == (-1, 2 | 4) and c.status() == (0, 0)
    got = run_plan(c, [16, 3], [1, 1], tables[:2], np.arange(8), [8, 2, 0], 2)        # head outside the ring: nothing is free
    assert list(got[0]) == [-1, 2 * 16 + 3] and list(got[3]) == [16, 4] and list(got[4]) == [0, 0, 1]
    assert c.status() == (-1, 8)


def test_plan_steps_in_a_graph():
    """Lengths and ring state in place: a captured step, replayed, serves one token after another; every page stays with
    one owner."""
    torch = torch_()
    B, page, n_pages = 5, 16, 40
    c = lib.PagedCache(1, 1, 64, page, n_pages, B, 8)
    ln, fs, tb, rg = ints(np.zeros(B)), ints([3, n_pages, 0]), ints(np.full((B, 8), -1)), ints(np.random.default_rng(1).permutation(n_pages))
    e = lambda n: torch.empty(n, dtype=torch.int32, device="cuda")  # noqa: E731
    out = lib.CachePlan(e(B), e(B), e(B + 1), ln, fs)
    c.plan(ln, None, tb, rg, fs, B, out=out)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        c.plan(ln, None, tb, rg, fs, B, out=out)
    seen = set()
    for step in range(1, 100):
        g.replay()
        torch.cuda.synchronize()
        assert ln.tolist() == [step + 1] * B and out.positions.tolist() == [step] * B
        seen.update(out.slots.tolist())
    assert len(seen) == 99 * B and min(seen) >= 0
    assert fs.tolist() == [(3 + 7 * B) % n_pages, n_pages - 7 * B, 0]


# ---------------------------------------------------------------- write

WRITES = [  # T, Hq, Hkv, D, page, rope, act, cache, with norm
    (1, 16, 2, 256, 16, 64, "f16", "f16", True), (1, 1, 1, 64, 16, 16, "bf16", "bf16", True),
    (3, 16, 2, 256, 16, 64, "bf16", "e4m3", True), (17, 5, 1, 64, 32, 64, "f16", "e4m3", True),
    (40, 32, 8, 128, 64, 128, "bf16", "bf16", False), (5, 9, 3, 128, 128, 48, "f16", "f16", True),
    (33, 64, 1, 64, 256, 0, "f16", "f16", True), (7, 6, 6, 256, 16, 256, "f16", "e4m3", False),
    (130, 14, 2, 64, 16, 32, "bf16", "e4m3", True), (300, 4, 4, 128, 16, 16, "f16", "f16", True)]


def write_case(T, Hq, Hkv, D, page, act, cache, seed, idle=0):
    torch = torch_()
    g = gen_of(seed)
    n_pages = -(-T // page) + 2
    x = randn(g, (T, 2 * Hq + 2 * Hkv, D), act, 2.0)          # the gate beside each query head, then k, then v
    q = x[:, :2 * Hq].view(T, Hq, 2, D)[:, :, 0]
    slots = torch.randperm(n_pages * page, generator=g, device="cuda")[:T].int()
    slots[T - idle:] = -1
    pool = randn(g, (n_pages, 2, Hkv, page, D), cache)        # keys and values of a page side by side
    d = dict(q=q, k=x[:, 2 * Hq:2 * Hq + Hkv], v=x[:, 2 * Hq + Hkv:], slots=slots, k_cache=pool[:, 0], v_cache=pool[:, 1],
             positions=torch.randint(0, 300000, (T,), generator=g, device="cuda", dtype=torch.int32),
             q_gamma=randn(g, (D,), act, 0.3), k_gamma=randn(g, (D,), act, 0.3))
    if cache == "e4m3":
        d["k_scale"] = torch.rand(Hkv, generator=g, device="cuda") * 0.02 + 0.005
        d["v_scale"] = torch.rand(Hkv, generator=g, device="cuda") * 0.02 + 0.005
    return d, n_pages


@pytest.mark.parametrize("T,Hq,Hkv,D,page,rope,act,cache,norm", WRITES)
def test_write_matches_the_oracle(T, Hq, Hkv, D, page, rope, act, cache, norm):
    torch = torch_()
    idle = T // 3
    d, n_pages = write_case(T, Hq, Hkv, D, page, act, cache, 10 * T + D, idle)
    if not norm:
        d["q_gamma"] = d["k_gamma"] = None
    theta, off, eps = 1e6, 1.0, 1e-5
    before = [f64(d["k_cache"]), f64(d["v_cache"])]
    c = lib.PagedCache(Hq, Hkv, D, page, n_pages, 1, 1, dtype=act, cache_dtype=cache, rope_dim=rope, rope_theta=theta,
                       gamma_offset=off, eps=eps)
    q = c.write(**d)
    torch.cuda.synchronize()
    assert c.status() == (0, 0)
    pos, slots = d["positions"].cpu().numpy(), d["slots"].cpu().numpy()
    u = U[act]
    y, size = O.norm_rope(f64(d["q"]), f64(d["q_gamma"]), pos, rope, theta, off, eps)
    tiny = 2.0 ** -25
    err = np.abs(f64(q) - y)
    assert (err <= u * np.abs(y) + 2.0 ** -20 * size + tiny).all(), err.max()
    yk, sk = O.norm_rope(f64(d["k"]), f64(d["k_gamma"]), pos, rope, theta, off, eps)
    for name, y, size, old, pool in (("k", yk, sk, before[0], d["k_cache"]), ("v", f64(d["v"]), np.abs(f64(d["v"])), before[1], d["v_cache"])):
        got = f64(pool)
        want, tol = old.copy(), np.zeros_like(old)
        for t in range(T):
            if slots[t] < 0:
                continue
            p, o = divmod(int(slots[t]), page)
            if cache == "e4m3":
                s = f64(d[name + "_scale"])[:, None]
                z = np.clip(y[t] / s, -448, 448)
                want[p, :, o] = z
                tol[p, :, o] = 2.0 ** -4 * np.abs(z) + 2.0 ** -10 + 2.0 ** -19 * size[t] / s
            else:
                want[p, :, o] = y[t]
                tol[p, :, o] = u * np.abs(y[t]) + 2.0 ** -20 * size[t] + tiny
        assert (np.abs(got - want) <= tol).all(), name         # rows that nothing wrote are bit for bit what they were
    if cache != "e4m3":                                        # a value goes into a cache of its own type as it is
        for t in np.flatnonzero(slots >= 0):
            p, o = divmod(int(slots[t]), page)
            assert torch.equal(d["v_cache"][p, :, o], d["v"][t])


def test_write_in_place_and_without_queries():
    torch = torch_()
    d, n_pages = write_case(9, 16, 2, 256, 16, "f16", "f16", 3)
    c = lib.PagedCache(16, 2, 256, 16, n_pages, 1, 1, rope_dim=64, gamma_offset=1.0)
    k0, v0 = d["k_cache"].clone(), d["v_cache"].clone()
    want = c.write(**d).clone()
    k1, v1 = d["k_cache"].clone(), d["v_cache"].clone()
    d["k_cache"].copy_(k0)
    d["v_cache"].copy_(v0)
    assert c.write(**{**d, "q": None}) is None
    assert torch.equal(d["k_cache"], k1) and torch.equal(d["v_cache"], v1)
    assert c.write(**d, q_out=d["q"]) is d["q"]
    assert torch.equal(d["q"], want)


def test_write_saturates_and_keeps_nan():
    torch = torch_()
    d, n_pages = write_case(2, 1, 1, 64, 16, "f16", "e4m3", 4)
    d["v"][0, 0, :4] = torch.tensor([6e4, -6e4, float("nan"), float("inf")], device="cuda", dtype=torch.float16)
    d["v_scale"][:] = 0.01
    c = lib.PagedCache(1, 1, 64, 16, n_pages, 1, 1, cache_dtype="e4m3")
    c.write(**d)
    p, o = divmod(int(d["slots"][0]), 16)
    got = d["v_cache"][p, 0, o, :4].float().tolist()
    assert got[0] == 448 and got[1] == -448 and got[2] != got[2] and got[3] == 448


def test_write_reports_slots_past_the_pool():
    torch = torch_()
    d, n_pages = write_case(4, 2, 1, 64, 16, "f16", "f16", 5)
    d["slots"][1], d["slots"][2] = n_pages * 16, -5
    k0 = d["k_cache"].clone()
    c = lib.PagedCache(2, 1, 64, 16, n_pages, 1, 1)
    c.write(**d)
    assert c.status() == (-1, 4) and c.status() == (0, 0)
    changed = (d["k_cache"] != k0).any(-1)[:, 0]              # [pages, page]
    assert set(changed.flatten().nonzero()[:, 0].tolist()) == {int(d["slots"][0]), int(d["slots"][3])}


def test_write_heads_far_apart():
    """Head strides of 2^29 elements: a step over a warp's heads passes 31 bits."""
    torch = torch_()
    T, H, D, far = 3, 5, 64, 1 << 29
    buf = torch.empty((H - 1) * far + T * D, dtype=torch.float16, device="cuda")
    g = gen_of(18)
    x = randn(g, (3, T, H, D), "f16")
    apart = buf.as_strided((T, H, D), (D, far, 1))
    c = lib.PagedCache(H, H, D, 16, 1, 1, 1, rope_dim=0)
    slots, positions = ints([0, 5, 15]), ints([0, 1, 2])
    kc, vc = randn(g, (1, H, 16, D), "f16"), randn(g, (1, H, 16, D), "f16")
    for far_q, far_k, far_v in ((1, 0, 0), (0, 1, 0), (0, 0, 1)):
        apart.copy_(x[0] if far_q else x[1] if far_k else x[2])
        q = c.write(apart if far_q else x[0], apart if far_k else x[1], apart if far_v else x[2], positions, slots, kc, vc,
                    q_out=apart if far_q else None)
        assert torch.equal(q, x[0])
        for t, slot in enumerate([0, 5, 15]):
            assert torch.equal(kc[0, :, slot], x[1, t]) and torch.equal(vc[0, :, slot], x[2, t])
    assert c.status() == (0, 0)


def test_write_far_positions():
    """Angles of positions up to 2^31 - 1 keep their fraction of a turn."""
    torch = torch_()
    d, n_pages = write_case(4, 2, 1, 128, 16, "bf16", "bf16", 6)
    d["positions"][:] = torch.tensor([2 ** 31 - 1, 16777217, 1048577, 0], device="cuda", dtype=torch.int32)
    c = lib.PagedCache(2, 1, 128, 16, n_pages, 1, 1, dtype="bf16", rope_dim=128, rope_theta=1e4)
    q = c.write(**{**d, "q_gamma": None, "k_gamma": None})
    y, size = O.norm_rope(f64(d["q"]), None, d["positions"].cpu().numpy(), 128, 1e4, 0, 0)
    # at 2^31 the product of position and frequency, 2^28 turns in fp64, is itself good to 2^-24 of a turn
    assert (np.abs(f64(q) - y) <= U["bf16"] * np.abs(y) + 2.0 ** -19 * size).all()


# ---------------------------------------------------------------- attend

def attend_case(lengths, Hq, Hkv, D, page, act, cache, seed, gate=True, width=None, gain=1.0):
    torch = torch_()
    g = gen_of(seed)
    B = len(lengths)
    held = [-(-n // page) for n in lengths]
    n_pages = sum(held) + 2
    width = width or max(held) + 1
    order = torch.randperm(n_pages, generator=g, device="cuda").tolist()
    tables = np.full((B, width), 2 ** 30, np.int32)           # entries past a request's pages are not looked at
    at = 0
    for b in range(B):
        tables[b, :held[b]] = order[at:at + held[b]]
        at += held[b]
    big = 8.0 if cache == "e4m3" else 1.0
    pool = randn(g, (n_pages, 2, Hkv, page, D), cache, big)
    raw = pool.view(torch.uint8) if cache == "e4m3" else pool.view(torch.int16)
    for b, n in enumerate(lengths):                           # NaN past the end of a request, and in pages of nobody
        if n % page:
            raw[tables[b, n // page], :, :, n % page:] = 0x7F if cache == "e4m3" else 0x7FFF
    raw[order[at]] = 0x7F if cache == "e4m3" else 0x7FFF
    x = randn(g, (B, Hq, 2, D), act, 1.5 * gain)              # the gate beside each query head
    d = dict(q=x[:, :, 0], tables=ints(tables), lengths=ints(lengths), k_cache=pool[:, 0], v_cache=pool[:, 1])
    if gate:
        d["gate"] = x[:, :, 1]
    if cache == "e4m3":
        d["k_scale"] = torch.rand(Hkv, generator=g, device="cuda") * 0.1 + 0.05
        d["v_scale"] = torch.rand(Hkv, generator=g, device="cuda") * 0.1 + 0.05
    return d, n_pages, width


def attend_check(d, out, Hq, Hkv, D, act, cache, scale=None):
    k, v = f64(d["k_cache"]), f64(d["v_cache"])
    if cache == "e4m3":
        k, v = k * f64(d["k_scale"])[:, None, None], v * f64(d["v_scale"])[:, None, None]
    lengths = d["lengths"].cpu().numpy()
    want, size, mag = O.attend(f64(d["q"]), d["tables"].cpu().numpy(), lengths, k, v, scale or D ** -0.5, f64(d.get("gate")))
    up = U["f16"] if cache == "e4m3" else U[act]
    delta = D * 2.0 ** -23 * mag
    tol = U[act] * np.abs(want) + size * (up + 2 * delta + (lengths[:, None, None] / 16 + 32) * 2.0 ** -23) + 2.0 ** -24
    got = f64(out)
    assert np.isfinite(want).all() and np.isfinite(got).all()
    bad = np.abs(got - want) > tol
    assert not bad.any(), (np.argwhere(bad)[:4], np.abs(got - want)[bad][:4], tol[bad][:4])
    assert (got[lengths == 0] == 0).all()


EDGES = [0, 1, 2, 15, 16, 17, 31, 33, 63, 64, 65, 127, 128, 129, 0, 191, 257, 1000]
ATTENDS = [  # lengths, Hq, Hkv, D, page, act, cache, gate
    (EDGES, 16, 2, 256, 16, "f16", "f16", True), (EDGES, 16, 2, 256, 16, "bf16", "e4m3", True),
    (EDGES, 32, 8, 128, 64, "bf16", "bf16", False), (EDGES, 5, 1, 64, 32, "f16", "e4m3", True),
    (EDGES, 9, 3, 128, 256, "f16", "f16", True), (EDGES, 64, 1, 64, 16, "f16", "f16", False),
    (EDGES, 17, 1, 256, 128, "bf16", "bf16", True), (EDGES, 32, 1, 256, 64, "f16", "e4m3", False),
    (EDGES, 6, 6, 64, 128, "bf16", "bf16", True), (EDGES, 14, 2, 128, 16, "bf16", "e4m3", True),
    ([1], 16, 2, 256, 16, "f16", "f16", True), ([0], 1, 1, 64, 16, "f16", "f16", False), ([0, 0, 0], 8, 4, 128, 16, "bf16", "e4m3", True),
    ([16], 24, 2, 256, 16, "bf16", "bf16", True), ([130], 16, 2, 256, 16, "f16", "f16", True),
    ([40001], 16, 2, 256, 16, "f16", "f16", True), ([70000, 3], 8, 1, 64, 64, "bf16", "e4m3", True),
    ([9000, 1, 0, 5000], 12, 4, 128, 32, "f16", "f16", False), ([20011], 40, 1, 64, 16, "bf16", "bf16", True),
    ([257] * 300, 8, 1, 64, 16, "f16", "f16", True), (list(range(1, 153)), 4, 2, 128, 16, "bf16", "bf16", False),
    ([700] * 37, 8, 8, 256, 256, "f16", "e4m3", True)]


@pytest.mark.parametrize("lengths,Hq,Hkv,D,page,act,cache,gate", ATTENDS, ids=[f"{len(a[0])}x{max(a[0])}-{a[1:]}" for a in ATTENDS])
def test_attend_matches_the_oracle(lengths, Hq, Hkv, D, page, act, cache, gate):
    torch = torch_()
    d, n_pages, width = attend_case(lengths, Hq, Hkv, D, page, act, cache, sum(lengths) + D, gate)
    c = lib.PagedCache(Hq, Hkv, D, page, n_pages, len(lengths), width, dtype=act, cache_dtype=cache)
    out = c.attend(**d)
    again = c.attend(**d)
    assert c.status() == (0, 0)
    attend_check(d, out, Hq, Hkv, D, act, cache)
    assert torch.equal(out, again)                            # sums in a fixed order


@pytest.mark.parametrize("page", [16, 32, 64, 128, 256])
@pytest.mark.parametrize("D,act,cache,Hq,Hkv", [(64, "f16", "e4m3", 9, 3), (64, "bf16", "bf16", 7, 1), (128, "bf16", "e4m3", 6, 2)])
def test_attend_copies_of_several_rows(D, act, cache, Hq, Hkv, page):
    """Rows of a line or less, copied by as much of a page as a stage holds: ends within a copy, within a page."""
    lengths = EDGES + [240, 241, 255, 256, 272, 273, 511, 513, 529]
    d, n_pages, width = attend_case(lengths, Hq, Hkv, D, page, act, cache, page + D, True)
    c = lib.PagedCache(Hq, Hkv, D, page, n_pages, len(lengths), width, dtype=act, cache_dtype=cache)
    out = c.attend(**d)
    assert c.status() == (0, 0)
    attend_check(d, out, Hq, Hkv, D, act, cache)
    long = lengths.index(529)
    d["tables"][long, 0], d["tables"][long, 1] = n_pages, -5  # read as zeros, whole copies of them
    out = c.attend(**d)
    assert c.status() == (-1, 4)
    attend_check(d, out, Hq, Hkv, D, act, cache)


@pytest.mark.parametrize("lengths", [EDGES, [9000, 0, 20011, 1, 16], [70001]], ids=["edges", "split", "one"])
@pytest.mark.parametrize("Hq,Hkv,D,page,act,cache,gate", [
    (32, 1, 128, 16, "bf16", "e4m3", True), (40, 2, 128, 32, "f16", "f16", True), (64, 1, 128, 64, "bf16", "bf16", False),
    (33, 1, 64, 16, "f16", "e4m3", True), (34, 2, 64, 128, "bf16", "bf16", True), (16, 1, 256, 16, "bf16", "e4m3", True),
    (24, 2, 256, 64, "f16", "f16", True), (48, 1, 256, 16, "f16", "e4m3", False)])
def test_attend_wide_groups(lengths, Hq, Hkv, D, page, act, cache, gate):
    """More query heads to a key-value head than a tile of eight."""
    torch = torch_()
    d, n_pages, width = attend_case(lengths, Hq, Hkv, D, page, act, cache, Hq + D, gate)
    c = lib.PagedCache(Hq, Hkv, D, page, n_pages, len(lengths), width, dtype=act, cache_dtype=cache)
    out = c.attend(**d)
    again = c.attend(**d)
    assert c.status() == (0, 0)
    attend_check(d, out, Hq, Hkv, D, act, cache)
    assert torch.equal(out, again)


def test_attend_calls_of_alternating_shapes_on_one_handle():
    torch = torch_()
    cases = [attend_case(n, 16, 2, 256, 16, "f16", "f16", 50 + i, width=400) for i, n in enumerate(([5000, 3, 700], [64] * 90, [1], [6000]))]
    n_pages = max(c[1] for c in cases)
    c = lib.PagedCache(16, 2, 256, 16, n_pages, 90, 400)
    full = []
    for d, n, _ in cases:                                     # pools of one size
        pool = torch.zeros((n_pages, 2, 2, 16, 256), dtype=torch.float16, device="cuda")
        pool[:n, 0], pool[:n, 1] = d["k_cache"], d["v_cache"]
        full.append({**d, "k_cache": pool[:, 0], "v_cache": pool[:, 1]})
    first = [c.attend(**d) for d in full]
    for d, o in zip(full, first):
        attend_check(d, o, 16, 2, 256, "f16", "f16")
    for _ in range(5):
        for d, o in zip(full, first):
            assert torch.equal(c.attend(**d), o)


def test_attend_scale_output_in_place_and_streams():
    torch = torch_()
    d, n_pages, width = attend_case([300, 20, 77], 16, 2, 256, 16, "bf16", "bf16", 9)
    c = lib.PagedCache(16, 2, 256, 16, n_pages, 3, width, dtype="bf16")
    want = c.attend(**d, scale=0.2)
    attend_check(d, want, 16, 2, 256, "bf16", "bf16", scale=0.2)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    out = c.attend(**d, scale=0.2, stream=side)
    side.synchronize()
    assert torch.equal(out, want)
    assert c.attend(**d, scale=0.2, out=d["q"]) is d["q"] and torch.equal(d["q"], want)


def test_attend_in_a_graph_with_lengths_that_grow():
    torch = torch_()
    d, n_pages, width = attend_case([900, 40, 513, 0], 16, 2, 256, 16, "f16", "f16", 11)
    for p in (d["k_cache"], d["v_cache"]):
        p.nan_to_num_(nan=0.25)
    c = lib.PagedCache(16, 2, 256, 16, n_pages, 4, width)
    d["lengths"].copy_(ints([100, 3, 0, 0]))
    out = c.attend(**d)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        c.attend(**d, out=out)
    for lengths in ([1, 0, 513, 0], [900, 40, 1, 0], [0, 0, 0, 0], [128, 39, 500, 0]):
        d["lengths"].copy_(ints(lengths))
        g.replay()
        attend_check(d, out, 16, 2, 256, "f16", "f16")


def test_attend_infinite_scores():
    """A score of -inf weighs nothing; a row of nothing else, or a score of +inf, gives NaN, as the formula does."""
    torch = torch_()
    d, n_pages, width = attend_case([200, 70, 70, 40], 8, 1, 64, 16, "f16", "f16", 13, gate=False)
    page = lambda b, j: (int(d["tables"][b, j // 16]), 0, j % 16)  # noqa: E731
    d["q"].abs_()
    for j in (0, 1, 2, 64, 65, 199):
        d["k_cache"][page(0, j)] = -float("inf")
    for j in range(70):
        d["k_cache"][page(1, j)] = -float("inf")
    d["k_cache"][page(2, 33)] = float("inf")
    c = lib.PagedCache(8, 1, 64, 16, n_pages, 4, width)
    out = c.attend(**d)
    assert torch.isnan(out[1]).all() and torch.isnan(out[2]).all() and torch.isfinite(out[0]).all()
    keep = {k: (v[::3] if k in ("q", "tables", "lengths") else v) for k, v in d.items()}
    k = f64(d["k_cache"])
    k[~np.isfinite(k)] = -1e9
    want, size, _ = O.attend(f64(keep["q"]), keep["tables"].cpu().numpy(), [200, 40], k, f64(d["v_cache"]), 0.125)
    assert (np.abs(f64(out[::3]) - want) <= 2.0 ** -9 * size).all()


def test_attend_reports_bad_pages_and_lengths():
    torch = torch_()
    d, n_pages, width = attend_case([40, 100, 50, 64], 16, 2, 128, 16, "f16", "f16", 15)
    d["tables"][1, 2], d["tables"][1, 4], d["tables"][3, 0] = n_pages, -1, 2 ** 31 - 1
    c = lib.PagedCache(16, 2, 128, 16, n_pages, 4, width)
    out = c.attend(**d)
    assert c.status() == (-1, 4)
    attend_check(d, out, 16, 2, 128, "f16", "f16")            # pages that are not there read as zeros
    d["lengths"][0], d["lengths"][1] = -3, 0
    out = c.attend(**d)
    assert c.status() == (-1, 2 | 4)
    d["lengths"][0] = 0
    attend_check(d, out, 16, 2, 128, "f16", "f16")


def test_attend_wait_that_runs_out_is_reported():
    """A copy that never comes: the call ends, the status says so, and the handle works again."""
    torch = torch_()
    for lengths in ([700, 90], [30000]):
        d, n_pages, width = attend_case(lengths, 16, 2, 256, 16, "f16", "f16", 16)
        c = lib.PagedCache(16, 2, 256, 16, n_pages, 2, width)
        want = c.attend(**d)
        c.set_wait(timeout_us=2000, skip_copy=True)
        c.attend(**d)
        s, f = c.status()
        assert s == -5 and f & 1, (s, f)
        assert c.status() == (0, 0)
        c.set_wait()
        assert torch.equal(c.attend(**d), want)
        assert c.status() == (0, 0)


def test_attend_offsets_past_32_bits():
    """Pools of more than 2^32 bytes: pages far apart."""
    torch = torch_()
    page, D, Hkv, stride = 16, 64, 1, 1 << 25
    pool = torch.empty(70 * stride, dtype=torch.float16, device="cuda")
    shape = (70, Hkv, page, D)
    kc = pool.as_strided(shape, (stride, page * D, D, 1))
    vc = pool.as_strided(shape, (stride, page * D, D, 1), page * D)
    g = gen_of(17)
    kc.copy_(randn(g, shape, "f16"))
    vc.copy_(randn(g, shape, "f16"))
    d = dict(q=randn(g, (2, 8, D), "f16"), tables=ints([[69, 3, 66, 1], [68, 0, 0, 0]]), lengths=ints([61, 9]), k_cache=kc, v_cache=vc)
    c = lib.PagedCache(8, Hkv, D, page, 70, 2, 4)
    attend_check(d, c.attend(**d), 8, Hkv, D, "f16", "f16")
    rows = randn(g, (2, 1, D), "f16")
    c.write(None, rows, rows, ints([0, 0]), ints([67 * 16 + 5, 2 * 16]), kc, vc)
    assert torch.equal(kc[67, :, 5], rows[0]) and torch.equal(vc[2, :, 0], rows[1])


def test_binding_refuses_wrong_tensors():
    torch = torch_()
    d, n_pages, width = attend_case([40], 16, 2, 128, 16, "f16", "f16", 15)
    c = lib.PagedCache(16, 2, 128, 16, n_pages, 1, width)
    for change in (dict(q=d["q"].bfloat16()), dict(q=d["q"][:, :8]), dict(tables=d["tables"].long()), dict(lengths=d["lengths"].cpu()),
                   dict(k_cache=d["k_cache"][1:]), dict(v_cache=d["v_cache"].transpose(2, 3)), dict(k_scale=torch.ones(3, device="cuda")),
                   dict(gate=d["gate"].float())):
        with pytest.raises(ValueError):
            c.attend(**{**d, **change})
    with pytest.raises(lib.MoeError):
        c.attend(**{**d, "k_scale": torch.ones(2, device="cuda")})      # scales for a cache that is not e4m3
    with pytest.raises(lib.MoeError):
        lib.PagedCache(16, 2, 96, 16, 4, 1, 1)
