"""Numbers at the edges of the paged cache's formats, against the float64 oracle: long flat tails under one high score,
scores so large that fp32 cannot hold a step between them.

Bounds. As in test_gpu_cache.py: a score is off by d = D 2^-23 sum|q k| scale, a weight by its rounding u(p), the sum over n
tokens by (n / 16 + 32) 2^-23, all relative to S = sum p |v|; the output by u(out) |out|. Weights of the second product are
fp16, as high as 2^15 for the highest score, unless the cache is bf16: those below 2^-14 have a half step of 2^-25, which is
2^-40 of the highest, so each value adds 2^-40 |v| times the highest weight, which is less than 1."""
import numpy as np
import pytest

import oracle.cache_oracle as O
from tests.test_gpu_cache import U, attend_case, dt, f64, gen_of, ints, randn, torch_
from w4a16_top_mixture_gb300 import build, lib

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    build.build()
    lib.load_library()


def one_request(k, v, act, cache, page=16):
    """A handle, and tables, lengths and pools of one request with the keys and values k, v [n, Hkv, D]."""
    torch = torch_()
    n, Hkv, D = k.shape
    pages = -(-n // page)

    def pool(x):
        x = torch.cat([x, torch.zeros(pages * page - n, Hkv, D, device="cuda")])
        return x.view(pages, page, Hkv, D).transpose(1, 2).contiguous().to(dt(cache))
    d = dict(tables=torch.arange(pages, dtype=torch.int32, device="cuda")[None], lengths=ints([n]), k_cache=pool(k), v_cache=pool(v))
    if cache == "e4m3":
        d["k_scale"], d["v_scale"] = torch.ones(Hkv, device="cuda"), torch.ones(Hkv, device="cuda")
    return d, lambda Hq: lib.PagedCache(Hq, Hkv, D, page, pages, 1, pages, dtype=act, cache_dtype=cache)


def reference(d, q, scale, gate=None):
    k, v = f64(d["k_cache"]), f64(d["v_cache"])
    if "k_scale" in d:
        k, v = k * f64(d["k_scale"])[:, None, None], v * f64(d["v_scale"])[:, None, None]
    return O.attend(f64(q), d["tables"].cpu().numpy(), d["lengths"].tolist(), k, v, scale, f64(gate))


TAILS = [(n, gap, sink, D, Hq, act, cache) for n, gap, sink in ((30000, 18.0, 0), (20000, 16.0, 19999), (20000, 20.0, 9000), (700, 14.0, 0))
         for D, Hq, act, cache in ((64, 8, "f16", "f16"), (64, 8, "bf16", "e4m3"), (64, 32, "f16", "e4m3"), (128, 16, "f16", "f16"),
                                   (128, 8, "bf16", "e4m3"), (128, 24, "bf16", "bf16"), (256, 4, "f16", "f16"), (256, 16, "bf16", "e4m3"))]


@pytest.mark.parametrize("n,gap,sink,D,Hq,act,cache", TAILS + [(131071, 18.0, 0, 64, 2, "f16", "f16"), (131071, 18.0, 0, 64, 2, "bf16", "e4m3")])
def test_attend_keeps_the_tail_under_one_high_score(n, gap, sink, D, Hq, act, cache):
    """One key `gap` above all others with a value of 0, so that the others make the whole output."""
    torch = torch_()
    g = gen_of(n + D + Hq)
    k, v = torch.randn(n, 1, D, generator=g, device="cuda") * 0.5, torch.randn(n, 1, D, generator=g, device="cuda") * 8 + 64
    k[..., 0] = 0
    k[sink], v[sink] = 0, 0
    k[sink, 0, 0] = gap
    d, handle = one_request(k, v, act, cache)
    scale = 0.125
    q = torch.randn(1, Hq, D, generator=g, device="cuda") * (0.5 * (64 / D) ** 0.5)
    q[..., 0] = 8                                             # scale * q . k = gap for the high key
    q = q.to(dt(act))
    c = handle(Hq)
    out = c.attend(q, scale=scale, **d)
    assert c.status() == (0, 0)
    want, size, mag = reference(d, q, scale)
    up = U["bf16"] if cache == "bf16" else U["f16"]
    lost = 0.0 if cache == "bf16" else 2.0 ** -40 * np.abs(f64(d["v_cache"])).sum((0, 2))     # [1, D]: one head of keys
    tol = U[act] * np.abs(want) + size * (up + 2 * D * 2.0 ** -23 * mag + (n / 16 + 32) * 2.0 ** -23) + lost + 2.0 ** -24
    err = np.abs(f64(out) - want)
    assert (err <= tol).all(), ((err / tol).max(), (err / size).max())


@pytest.mark.parametrize("act,cache", [("f16", "f16"), ("bf16", "e4m3"), ("bf16", "bf16")])
@pytest.mark.parametrize("high", [2.0 ** 12, 2.0 ** 19, 2.0 ** 22, 2.0 ** 25, -(2.0 ** 22), -(2.0 ** 25)])
def test_attend_scores_past_a_step_of_fp32(high, act, cache):
    """Scores of `high` up to 2^28, equal for two or all of the keys: the mean of those keys' values."""
    torch = torch_()
    g = gen_of(3)
    n, D, Hq = 900, 64, 5
    k, v = torch.zeros(n, 1, D, device="cuda"), torch.randn(n, 1, D, generator=g, device="cuda") * 4
    k[..., 0] = 16 if high < 0 else -16
    k[300, 0, 0] = k[777, 0, 0] = 16
    d, handle = one_request(k, v, act, cache)
    q = torch.zeros(1, Hq, D, device="cuda")
    q[0, :, 0] = torch.tensor([1.0, 1.5, 1.25, 7.0, 3.0], device="cuda")
    out = handle(Hq).attend(q.to(dt(act)), scale=high / 16, **d)
    v = f64(d["v_cache"]).reshape(-1, D)[:n]
    mine = v if high < 0 else v[[300, 777]]
    want, size = mine.mean(0), np.abs(mine).mean(0)
    up = U["bf16"] if cache == "bf16" else U["f16"]
    assert (np.abs(f64(out)[0] - want) <= U[act] * np.abs(want) + size * (up + (n / 16 + 32) * 2.0 ** -23) + 2.0 ** -24).all()


@pytest.mark.parametrize("D,Hq", [(64, 3), (128, 16), (256, 8), (256, 17)])
@pytest.mark.parametrize("e", [-125, -110, -60, -3, 0, 40, 99, 100, 101, 110, 124])
def test_attend_bf16_queries_of_any_size_over_e4m3(e, D, Hq):
    """Queries around 2^e with scales that bring the scores back to a few units: the products run in fp16, for which the
    queries are scaled by a power of two. Elements below 2^-14 of a head's largest lose bits there: half a step is 2^-25,
    so a score is off by 2^-25 max|q| sum|k| scale more."""
    torch = torch_()
    g = gen_of(e + D)
    n = 333
    k, v = (torch.randn(n, 1, D, generator=g, device="cuda") * 8 for _ in range(2))
    d, handle = one_request(k, v, "bf16", "e4m3")
    half = e // 2
    d["k_scale"].fill_(0.125 * 2.0 ** -half)
    scale = D ** -0.5 * 2.0 ** (half - e)
    q = (torch.randn(1, Hq, D, generator=g, device="cuda").clamp(-3.5, 3.5) * 1.1).to(torch.bfloat16).double() * 2.0 ** e
    q = q.to(torch.bfloat16)
    c = handle(Hq)
    out = c.attend(q, scale=scale, **d)
    want, size, mag = reference(d, q, scale)
    keys = np.abs(f64(d["k_cache"])).sum(-1).max() * f64(d["k_scale"])[0]
    delta = D * 2.0 ** -23 * mag + 2.0 ** -25 * np.abs(f64(q)).max(-1, keepdims=True) * keys * scale
    tol = U["bf16"] * np.abs(want) + size * (U["f16"] + 2 * delta + (n / 16 + 32) * 2.0 ** -23) + 2.0 ** -24
    err = np.abs(f64(out) - want)
    assert (err <= tol).all(), ((err / tol).max(), (err / size).max())


@pytest.mark.parametrize("n", [1, 40000])
@pytest.mark.parametrize("D,Hq,act,cache", [(64, 8, "bf16", "bf16"), (64, 2, "bf16", "e4m3"), (256, 24, "bf16", "bf16"), (128, 9, "f16", "f16")])
def test_attend_gates_far_from_zero(n, D, Hq, act, cache):
    """exp(-|gate|) in fp32 is off by 2 + 1.17 |gate| steps, 2^-16 at its smallest normal value, then by steps of 2^-149; all
    tokens hold one value, so the output is that value times the sigmoid."""
    torch = torch_()
    g = gen_of(D + n)
    v = torch.full((n, 1, D), 448.0 if cache == "e4m3" else 1e4, device="cuda")
    d, handle = one_request(torch.randn(n, 1, D, generator=g, device="cuda"), v, act, cache)
    if cache == "e4m3":
        d["v_scale"].fill_(20.0)
    gates = [-float("inf"), -110, -104, -100, -95, -90, -89, -88.5, -88, -87.5, -87, -80, -40, -11, -3, 0, 2, 17, 87, 88, 89, 104, float("inf")]
    gate = torch.tensor(gates, device="cuda").repeat(-(-Hq * D // len(gates)))[:Hq * D].view(1, Hq, D).to(dt(act))
    q = randn(g, (1, Hq, D), act)
    out = handle(Hq).attend(q, gate=gate, **d)
    y = float(f64(d["v_cache"])[0, 0, 0, 0]) * (20.0 if cache == "e4m3" else 1.0)
    x = f64(gate)
    want = y * np.exp(np.minimum(x, 0)) / (1 + np.exp(-np.abs(x)))
    up = U["bf16"] if cache == "bf16" else U["f16"]
    least = 2.0 ** -134 if act == "bf16" else 2.0 ** -25
    tol = want * (U[act] + up + (n / 16 + 32) * 2.0 ** -23 + 2.0 ** -16) + 3 * y * 2.0 ** -149 + least
    err = np.abs(f64(out) - want)
    assert (err <= tol).all(), (x[err > tol], f64(out)[err > tol], want[err > tol])


@pytest.mark.parametrize("act", ["f16", "bf16"])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_write_codes_are_those_of_an_fp32_division(D, act):
    """Code for code, over scales from fp32's smallest to its largest; the same for keys that nothing norms or turns."""
    torch = torch_()
    scales = [1e-45, 1e-39, 2.0 ** -130, 1.3e-38, 1e-30, 3e-20, 6e-20, 0.0123, 0.7, 1.0, 0.0137, 1.7e19, 2e19, 1e30, 3e38]
    T, H, page = 400, len(scales), 32
    g = gen_of(D)
    s = torch.tensor(scales, device="cuda")
    near = (torch.randn(2, T, H, D, generator=g, device="cuda").double() * 100 * s.double()[:, None]).to(dt(act))
    wild = (torch.randn(2, T, H, D, generator=g, device="cuda").double()
            * 2.0 ** (torch.rand(2, T, H, D, generator=g, device="cuda") * 260 - 134).double()).to(dt(act))
    x = torch.where(torch.rand(2, T, H, D, generator=g, device="cuda") < 0.5, near, wild)
    x[:, :5, :, 7:] = torch.tensor([0.0, -0.0, float("inf"), -float("inf"), float("nan")], device="cuda").to(dt(act))[None, :, None, None]
    pool = torch.zeros(2, -(-T // page), H, page, D, device="cuda").to(dt("e4m3"))
    c = lib.PagedCache(H, H, D, page, pool.shape[1], 1, 1, dtype=act, cache_dtype="e4m3")
    slots = torch.randperm(T, generator=g, device="cuda").int()
    c.write(None, x[0], x[1], slots, slots, pool[0], pool[1], k_scale=s, v_scale=s)
    got = pool.float().transpose(2, 3).reshape(2, -1, H, D)[:, slots.long()].cpu()
    want = (x.float().cpu() / s.cpu()[:, None]).clamp(-448, 448).to(torch.float8_e4m3fn).float()
    assert ((got == want) | (got.isnan() & want.isnan())).all()


@pytest.mark.parametrize("n,shortest,longest,empty,Hq,Hkv,D,page,act,cache,gate", [
    (128, 512, 16000, 5, 16, 2, 256, 16, "f16", "f16", True), (61, 1, 9000, 1, 32, 8, 128, 64, "bf16", "bf16", False),
    (256, 300, 5000, 11, 16, 2, 256, 32, "bf16", "e4m3", True)])
def test_attend_full_batches_with_empty_slots(n, shortest, longest, empty, Hq, Hkv, D, page, act, cache, gate):
    """A server's batches, every request compared, with a reference in 64 bits on the GPU. Nothing but the rows past a
    request's end and the page that nobody holds is NaN."""
    torch = torch_()
    lengths = [int(round(shortest * (longest / shortest) ** (i / (n - 1)))) for i in range(n)]
    lengths[:empty] = [0] * empty
    lengths = [lengths[i] for i in np.random.default_rng(n).permutation(n)]
    d, n_pages, width = attend_case(lengths, Hq, Hkv, D, page, act, cache, n, gate)
    c = lib.PagedCache(Hq, Hkv, D, page, n_pages, n, width, dtype=act, cache_dtype=cache)
    out = c.attend(**d)
    assert c.status() == (0, 0)
    one = torch.ones(Hkv, device="cuda")
    ks, vs = (d.get(x, one).double()[:, None, None] for x in ("k_scale", "v_scale"))
    up = U["bf16"] if cache == "bf16" else U["f16"]
    for b, m in enumerate(lengths):
        if not m:
            assert (out[b] == 0).all()
            continue
        ids = d["tables"][b, :-(-m // page)].long()
        k, v = (torch.stack([pool[i] for i in ids.tolist()]).transpose(0, 1).reshape(Hkv, -1, D)[:, :m].double() for pool in (d["k_cache"], d["v_cache"]))
        k, v = k * ks, v * vs
        q = d["q"][b].double().view(Hkv, -1, D)
        p = torch.softmax(q @ k.transpose(1, 2) * D ** -0.5, -1)
        mag = (q.abs() @ k.abs().transpose(1, 2)).amax(-1, keepdim=True) * D ** -0.5
        want, size = p @ v, p @ v.abs()
        if gate:
            sg = torch.sigmoid(d["gate"][b].double()).view(Hkv, -1, D)
            want, size = want * sg, size * sg
        tol = U[act] * want.abs() + size * (up + 2 * D * 2.0 ** -23 * mag + (m / 16 + 32) * 2.0 ** -23) + 2.0 ** -24
        assert ((out[b].double().view(Hkv, -1, D) - want).abs() <= tol).all(), (b, m)
