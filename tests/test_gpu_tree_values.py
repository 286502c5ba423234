"""Values that are not finite, or large, in the attention of several new tokens: in items that are split over CTAs, in rows that
see nothing, at the ends of the types' ranges, and the time that a call takes over them.

The reference is the formula in float64 on the GPU, a request at a time; its bound is that of test_gpu_tree.py."""
import pytest

from test_gpu_cache import U, ints, torch_
from test_gpu_tree import tree_case
from w4a16_top_mixture_gb300 import build, lib

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    build.build()
    lib.load_library()


def cache_of(d, n_pages, width, Hq, Hkv, D, page, act, cache, most):
    return lib.PagedCache(Hq, Hkv, D, page, n_pages, len(d["lengths"]), width, dtype=act, cache_dtype=cache, max_new=most)


def reference(d, page, scale):
    """(out, size, mag, seen) of the rows of all requests: the masked softmax in float64, where a weight of a value that a row
    does not see is no product at all. Of values that are not finite a row gets their sum, whatever their weights."""
    torch = torch_()
    q = d["q"].double()
    rows, Hq, D = q.shape
    k_pool, v_pool = d["k_cache"].double(), d["v_cache"].double()
    Hkv = k_pool.shape[1]
    out, size = torch.zeros_like(q), torch.zeros_like(q)
    mag, seen = torch.zeros(rows, Hq, 1, device="cuda").double(), torch.zeros(rows, 1, 1, device="cuda").double()
    starts = d["starts"].tolist()
    for b, n in enumerate(d["lengths"].tolist()):
        lo, hi = starts[b], starts[b + 1]
        m, pos = hi - lo, torch.arange(n, device="cuda")
        if m == 0 or ("slots" in d and int(d["slots"][lo]) < 0):
            continue
        new = torch.arange(m, device="cuda")
        sees = torch.ones(m, n, dtype=torch.bool, device="cuda")
        sees[:, n - m:] = (d["masks"][lo:hi][:, new // 64] >> (new % 64) & 1).bool() if "masks" in d else new[:, None] >= new
        seen[lo:hi, 0, 0] = sees.sum(1).double()
        pages = d["tables"][b].long()[pos // page]
        k, v = k_pool[pages, :, pos % page], v_pool[pages, :, pos % page]          # [n, Hkv, D]
        if "k_scale" in d:
            k, v = k * d["k_scale"].double()[:, None], v * d["v_scale"].double()[:, None]
        s = torch.zeros(m, Hq, n, device="cuda").double()
        for h in range(Hq):
            g = h // (Hq // Hkv)
            s[:, h] = q[lo:hi, h] @ k[:, g].T * scale
            mag[lo:hi, h, 0] = torch.where(sees, q[lo:hi, h].abs() @ k[:, g].abs().T, 0.0).amax(1) * abs(scale)
            p = torch.softmax(s[:, h].masked_fill(~sees, -float("inf")), 1)
            p = torch.where(sees.any(1, keepdim=True), p, 0.0)
            fine = torch.where(v[:, g].isfinite(), v[:, g], 0.0)
            y, z = p @ fine, p @ fine.abs()
            of = lambda what: sees.double() @ what.double() > 0                    # noqa: E731
            up, down, none = of(v[:, g] == float("inf")), of(v[:, g] == -float("inf")), of(v[:, g].isnan())
            y = torch.where(up, float("inf"), torch.where(down, -float("inf"), y))
            out[lo:hi, h], size[lo:hi, h] = torch.where(none | (up & down), float("nan"), y), z
    if "gate" in d:
        sg = torch.sigmoid(d["gate"].double())
        out, size = torch.where(seen > 0, out * sg, 0.0), size * sg
    return out, size, mag, seen


def check(d, got, page, act, cache, scale=None):
    torch = torch_()
    rows, D = int(d["starts"][-1]), d["q"].shape[2]
    want, size, mag, seen = (t[:rows] for t in reference(d, page, D ** -0.5 if scale is None else scale))
    got = got[:rows].double()
    up = U["f16"] if cache == "e4m3" else U[act]
    tol = U[act] * want.abs() + size * (up + 2 * D * 2.0 ** -23 * mag + 2.0 ** -21 * mag + (seen / 16 + 232) * 2.0 ** -23) + 2.0 ** -24
    ok = want.isfinite()
    assert torch.equal(got.isnan(), want.isnan())
    assert (got[want.isinf()] == want[want.isinf()]).all()
    bad = ((got - want).abs() > tol) & ok
    assert not bad.any(), (bad.nonzero()[:4], (got - want).abs()[bad][:4], tol[bad][:4])
    return want


def spoil(d, b, older, page, where):
    """where: (new token, element, value) for request b's values, key-value head 0."""
    for j, x, value in where:
        at = older + j
        d["v_cache"][int(d["tables"][b, at // page]), 0, at % page, x] = value


INF = float("inf")
ODD = [(2, 256, 16, "f16", "f16"), (2, 64, 32, "f16", "e4m3"), (2, 128, 64, "bf16", "bf16"), (2, 256, 16, "bf16", "e4m3"),
       (4, 64, 16, "bf16", "bf16"), (2, 128, 16, "f16", "e4m3")]


@pytest.mark.parametrize("masks", ["tree", None])
@pytest.mark.parametrize("Hq,D,page,act,cache", ODD)
@pytest.mark.parametrize("reqs", [[(6000, 150, 0)], [(30000, 150, 0)], [(2000 + 77 * i, 150 - i, 0) for i in range(9)]],
                         ids=["parts of a few tiles", "groups of parts", "two or three parts"])
def test_values_that_are_not_finite_in_items_of_several_parts(reqs, Hq, D, page, act, cache, masks):
    """New tokens with NaN or infinities lie in two to four tiles, so on either side of a border between CTAs in some item."""
    torch = torch_()
    d, n_pages, width = tree_case(reqs, Hq, 1, D, page, act, cache, D + len(reqs), len(reqs) > 1, masks, 3)
    nan = [float("nan")]
    for b, (older, n, _) in enumerate(reqs):
        few = [(0, 5, nan[0]), (n // 2, 9, nan[0]), (n - 1, 7, nan[0]), (n - 1, D - 1, nan[0])]
        if cache != "e4m3":
            few += [(1, 11, INF), (63, 12, -INF), (64, 13, INF), (n - 2, 13, -INF), (n - 1, 14, INF), (n - 3, 14, INF)]
        spoil(d, b, older, page, few if b % 2 == 0 else few[2:])
    c = cache_of(d, n_pages, width, Hq, 1, D, page, act, cache, 150)
    out = c.attend_tree(**d)
    assert c.status() == (0, 0)
    want = check(d, out, page, act, cache)
    assert not want.isfinite().all() and want.isfinite().any()
    assert torch.equal(c.attend_tree(**d).view(torch.int16), out.view(torch.int16))


@pytest.mark.parametrize("Hq,Hkv,D,page,act,cache", [(16, 2, 256, 16, "f16", "f16"), (32, 8, 128, 64, "bf16", "bf16"), (8, 2, 64, 16, "f16", "e4m3")])
@pytest.mark.parametrize("masks", ["tree", None])
@pytest.mark.parametrize("kind", ["one", "all NaN", "all infinite"])
def test_values_that_are_not_finite_do_not_hold_up_the_others(Hq, Hkv, D, page, act, cache, masks, kind):
    """One request of a batch of chunks has them. No wait of the call comes near 2 ms, and the other requests get the same bytes."""
    torch = torch_()
    if cache == "e4m3" and kind == "all infinite":
        pytest.skip("e4m3 has no infinities")
    reqs = [(250 * i, 256, 0) for i in range(12)]
    d, n_pages, width = tree_case(reqs, Hq, Hkv, D, page, act, cache, 3, False, masks, 4)
    c = cache_of(d, n_pages, width, Hq, Hkv, D, page, act, cache, 256)
    base = c.attend_tree(**d)
    older, at = reqs[5][0], d["tables"][5].long()
    if kind == "one":
        spoil(d, 5, older, page, [(0, 3, float("nan") if cache == "e4m3" else INF)])
    else:
        pos = torch.arange(older, older + 256, device="cuda")
        d["v_cache"][at[pos // page], :, pos % page] = torch.tensor(float("nan") if kind == "all NaN" else INF, device="cuda").to(d["v_cache"].dtype)
    c.set_wait(timeout_us=2000)
    out = c.attend_tree(**d)
    assert c.status() == (0, 0)
    s = d["starts"].tolist()
    assert torch.equal(out[:s[5]], base[:s[5]]) and torch.equal(out[s[6]:], base[s[6]:])
    one = {**d, "q": d["q"][s[5]:s[6]], "starts": ints([0, 256]), "tables": d["tables"][5:6], "lengths": d["lengths"][5:6],
           "slots": d["slots"][s[5]:s[6]]}
    if masks:
        one["masks"] = d["masks"][s[5]:s[6]]
    want = check(one, out[s[5]:s[6]], page, act, cache)
    assert not want.isfinite().all()


@pytest.mark.parametrize("Hq,D,page,act,cache", ODD[:4])
@pytest.mark.parametrize("reqs", [[(37, 6, 1), (0, 20, 0), (90, 4, 0)], [(0, 256, 0)]], ids=["short", "several parts"])
def test_rows_that_see_nothing_give_zero_whatever_their_gate(reqs, Hq, D, page, act, cache):
    """0 without a token, not 0 times the gate's sigmoid: rows of refused and of left-out requests, and rows whose masks are empty
    in requests without older tokens, under gates that are NaN."""
    torch = torch_()
    d, n_pages, width = tree_case(reqs, Hq, 1, D, page, act, cache, D, True, "any", 4, 2)
    c = cache_of(d, n_pages, width, Hq, 1, D, page, act, cache, 256)
    base = c.attend_tree(**d)
    rows = int(d["starts"][-1])
    empty = (reference(d, page, 1.0)[3] == 0).view(-1)
    assert empty[:rows].any() and not empty[:rows].all()
    d["gate"] = torch.where(empty[:, None, None], float("nan"), d["gate"].float()).to(d["gate"].dtype)
    got = c.attend_tree(**d)
    assert c.status() == (0, 0)
    assert torch.equal(got[:rows], base[:rows]) and (got[:rows][empty[:rows]] == 0).all()
    d["lengths"][len(reqs) - 1] = 1                            # fewer than its new ones: left out
    d["gate"].fill_(float("nan"))
    got = c.attend_tree(**d)
    assert c.status() == (-1, 2)
    assert (got[int(d["starts"][-2]):rows] == 0).all()


@pytest.mark.parametrize("older", [30, 3000])
@pytest.mark.parametrize("Hq,D,page,act,cache", [ODD[0], ODD[2], ODD[4]])
def test_rows_whose_scores_are_all_minus_infinity_give_zero(older, Hq, D, page, act, cache):
    """Whatever their values and gates; rows of another request in the batch, and of other heads, are as they were."""
    torch = torch_()
    d, n_pages, width = tree_case([(older, 5, 0), (60, 3, 0)], 2 * Hq, 2, D, page, act, cache, 7, True, "tree", 1)
    d["q"][..., 0] = 1.0
    c = lib.PagedCache(2 * Hq, 2, D, page, n_pages, 2, width, dtype=act, cache_dtype=cache, max_new=5)
    base = c.attend_tree(**d)
    pos = torch.arange(older + 5, device="cuda")
    pages = d["tables"][0].long()[pos // page]
    d["k_cache"][pages, 0, pos % page, 0] = -INF
    d["v_cache"][pages[:7], 0, pos[:7] % page, 4] = INF
    d["gate"][1, 0, 9] = float("nan")
    got = c.attend_tree(**d)
    assert c.status() == (0, 0)
    assert (got[:5, :Hq] == 0).all()
    assert torch.equal(got[5:], base[5:]) and torch.equal(got[:5, Hq:], base[:5, Hq:])


@pytest.mark.parametrize("older,size", [(370, 2.0 ** 100), (370, 2.0 ** 117), (370, -2.0 ** 117), (3000, 2.0 ** 114)])
def test_large_bf16_values_under_scores_that_rise(older, size):
    """A row's base may stay below its highest score by a factor of 2^8; its weights stay at 1 or below all the same, so that the
    sum over the tokens is within fp32's range where n times the largest value is: 373 2^117 < 2^126, 3003 2^114 < 2^126."""
    torch = torch_()
    D, page = 128, 64
    d, n_pages, width = tree_case([(older, 3, 0)], 4, 1, D, page, "bf16", "bf16", 11, False, None)
    n = older + 3
    pos = torch.arange(n, device="cuda")
    pages, off = d["tables"][0].long()[pos // page], pos % page
    d["q"].zero_()
    d["q"][..., 0] = 1.0
    d["k_cache"][pages, 0, off] = 0.0
    d["k_cache"][pages, 0, off, 0] = torch.where(pos < 128, 0.0, 5.4375).bfloat16()    # 2^7.84 in weights
    d["v_cache"][pages, 0, off] = torch.randn(n, D, device="cuda", generator=torch.Generator("cuda").manual_seed(1)).clamp(-1, 1).bfloat16()
    d["v_cache"][pages, 0, off] *= size
    d["v_cache"][pages, 0, off, 3] = size
    c = cache_of(d, n_pages, width, 4, 1, D, page, "bf16", "bf16", 3)
    out = c.attend_tree(**d, scale=1.0)
    assert c.status() == (0, 0)
    check(d, out, page, "bf16", "bf16", 1.0)
    assert (out[:3, :, 3].double() - size).abs().max() <= 2.0 ** -6 * abs(size)


FULL = [([(500 + 60 * i, 5 + i % 12, 0) for i in range(128)], (16, 2, 256, 16, "bf16", "e4m3")), ([(250 * i, 256, 0) for i in range(24)], (16, 2, 128, 64, "bf16", "bf16")),
        ([(40 * i % 900, 1 + i % 40, i % 11 == 5) for i in range(300)], (16, 2, 256, 16, "f16", "f16")), ([(80 * 2 ** i % 8100, 64, 0) for i in range(16)], (16, 2, 256, 16, "f16", "f16")),
        ([(0 if i % 7 else 3000, (256, 1, 9, 64, 0)[i % 5], i % 13 == 4) for i in range(90)], (8, 2, 64, 16, "f16", "e4m3")),
        ([(1000 + i, 1, 0) for i in range(200)] + [(2000, 256, 0), (0, 200, 0)], (16, 2, 128, 32, "f16", "e4m3"))]


@pytest.mark.parametrize("masks", ["tree", None])
@pytest.mark.parametrize("reqs,shape", FULL, ids=["trees, e4m3", "chunks", "300 mixed", "ragged", "mixed steps, e4m3", "decoding and prompts, e4m3"])
def test_every_request_of_long_batches(reqs, shape, masks):
    """Decoding requests, drafts, chunks, refused and empty ones in one batch, all of them compared."""
    torch = torch_()
    Hq, Hkv, D, page, act, cache = shape
    d, n_pages, width = tree_case(reqs, Hq, Hkv, D, page, act, cache, len(reqs), True, masks, 4, 3)
    c = cache_of(d, n_pages, width, Hq, Hkv, D, page, act, cache, 256)
    out = torch.full_like(d["q"], 7.0).contiguous()
    c.attend_tree(**d, out=out)
    assert c.status() == (0, 0)
    check(d, out, page, act, cache)
    assert (out[int(d["starts"][-1]):] == 7.0).all()


@pytest.mark.parametrize("older", [0, 5000])
@pytest.mark.parametrize("Hq,D,page,act,cache", [(2, 64, 32, "bf16", "e4m3"), (5, 256, 16, "bf16", "bf16"), (3, 128, 16, "f16", "f16")])
def test_gates_far_from_zero(older, Hq, D, page, act, cache):
    """exp(-|gate|) in fp32 is off by 2 + 1.17 |gate| steps, 2^-16 at its smallest normal value, then by steps of 2^-149; all tokens
    hold one value, so the output is that value times the sigmoid. One reciprocal of four factors adds a few steps of 2^-23."""
    torch = torch_()
    d, n_pages, width = tree_case([(older, 6, 0)], Hq, 1, D, page, act, cache, D, True, None)
    n = older + 6
    pos = torch.arange(n, device="cuda")
    value = 448.0 if cache == "e4m3" else 1e4
    d["v_cache"][d["tables"][0].long()[pos // page], 0, pos % page] = torch.tensor(value, device="cuda").to(d["v_cache"].dtype)
    y = float(torch.tensor(value).to(d["v_cache"].dtype))
    if cache == "e4m3":
        d["v_scale"].fill_(20.0)
        y *= 20.0
    gates = torch.tensor([-INF, -110, -104, -100, -95, -90, -89, -88.5, -88, -87.5, -87, -80, -40, -11, -3, 0, 2, 17, 87, 88, 89, 104, INF], device="cuda")
    shape = d["gate"].shape
    d["gate"] = gates.repeat(-(-d["gate"].numel() // len(gates)))[:d["gate"].numel()].view(shape).to(d["gate"].dtype)
    c = cache_of(d, n_pages, width, Hq, 1, D, page, act, cache, 6)
    out = c.attend_tree(**d).double()
    x = d["gate"].double()
    want = y * torch.exp(x.clamp(max=0)) / (1 + torch.exp(-x.abs()))
    up = U["f16"] if cache == "e4m3" else U[act]
    least = 2.0 ** -134 if act == "bf16" else 2.0 ** -25
    tol = want * (U[act] + up + (n / 16 + 232) * 2.0 ** -23 + 2.0 ** -16) + 3 * y * 2.0 ** -149 + least
    err = (out - want).abs()
    assert (err <= tol).all(), (x[err > tol][:9], out[err > tol][:9], want[err > tol][:9])
