"""What the calls for several new tokens report and refuse, and batches long enough that every ring, barrier and join of the
attention is used many times."""
import numpy as np
import pytest

from test_gpu_cache import gen_of, ints, randn, torch_
from test_gpu_tree import SHAPES, oracle_of, tree_case, tree_check
from w4a16_top_mixture_gb300 import build, lib

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    build.build()
    lib.load_library()


@pytest.mark.parametrize("shape", [0, 1, 2])
def test_attend_tree_reports_a_wait_that_runs_out(shape):
    """The first copy of the first CTA is left out: the call ends, says so, and the next ones compute nothing until it was
    read; then all is as before."""
    torch = torch_()
    Hq, Hkv, D, page, act, cache, gate = SHAPES[shape]
    d, n_pages, width = tree_case([(700, 9, 0), (3000, 5, 0)], Hq, Hkv, D, page, act, cache, 21, gate)
    c = lib.PagedCache(Hq, Hkv, D, page, n_pages, 2, width, dtype=act, cache_dtype=cache, max_new=9)
    want = c.attend_tree(**d)
    assert c.status() == (0, 0)
    c.set_wait(timeout_us=2000, skip_copy=True)
    c.attend_tree(**d)
    out = torch.full_like(want, 5.0)
    c.attend_tree(**d, out=out)                                # not reported yet
    status, flags = c.status()
    assert status == -5 and flags & 1 and (out == 5.0).all()
    c.set_wait()
    assert torch.equal(c.attend_tree(**d), want) and c.status() == (0, 0)


def test_calls_before_a_reserve_and_a_second_reserve():
    c = lib.PagedCache(1, 1, 64, 16, 8, 4, 2)
    i = lambda *s: ints(np.zeros(s))  # noqa: E731
    q = torch_().zeros(2, 1, 64, device="cuda").half()
    kc = torch_().zeros(c.pool_shape, device="cuda").half()
    for call in (lambda: c.tree(i(2), i(2), i(1), words=1), lambda: c.attend_tree(q, i(2), i(1, 2), i(1), kc, kc),
                 lambda: c.keep(i(1), i(1), i(1, 2), i(8), i(3), c.pools([kc])),
                 lambda: c.fork(i(1), i(1), i(1), i(1, 2), i(8), i(3), i(8), c.pools([kc]))):
        with pytest.raises(lib.MoeError) as e:
            call()
        assert e.value.status == -3
    assert c.lib.moe_cache_reserve(c.h, 0) == -2 and c.lib.moe_cache_reserve(c.h, 257) == -2
    assert c.lib.moe_cache_reserve(c.h, 8) == 0 and c.lib.moe_cache_reserve(c.h, 8) == -1
    with pytest.raises(ValueError):
        c.keep(i(1), i(1), i(1, 2), i(8), i(3), lib.PagedCache(1, 1, 64, 16, 8, 4, 2).pools([kc]))


LONG = [([(80 * 2 ** i % 8100, 64, 0) for i in range(16)], 0), ([(500 + 60 * i, 5 + i % 12, 0) for i in range(128)], 1),
        ([(250 * i, 256, 0) for i in range(24)], 2), ([(4032, 64, 0)] * 20, 3), ([(2000 + i, 1 + i % 3, 0) for i in range(300)], 10),
        ([(60000, 33, 0)], 4), ([(30000, 64, 0), (7, 64, 0)], 7)]


@pytest.mark.parametrize("reqs,shape", LONG, ids=lambda x: str(x)[:24])
def test_long_batches_repeat_and_agree_with_the_oracle_in_places(reqs, shape):
    """The same call twelve times: the same bytes, nothing reported; two requests of it against the oracle."""
    torch = torch_()
    Hq, Hkv, D, page, act, cache, gate = SHAPES[shape]
    words = -(-max(n for _, n, _ in reqs) // 64)
    d, n_pages, width = tree_case(reqs, Hq, Hkv, D, page, act, cache, 31, gate, "tree", words)
    c = lib.PagedCache(Hq, Hkv, D, page, n_pages, len(reqs), width, dtype=act, cache_dtype=cache, max_new=64 * words)
    want = c.attend_tree(**d)
    for _ in range(11):
        assert torch.equal(c.attend_tree(**d), want)
    assert c.status() == (0, 0)
    starts = d["starts"].tolist()
    small = sorted(range(len(reqs)), key=lambda b: reqs[b][0] * reqs[b][1])
    for b in {small[0], small[len(small) // 3]}:
        if reqs[b][0] * reqs[b][1] * Hq > 20_000_000:
            continue
        rows = slice(starts[b], starts[b + 1])
        one = {k: v for k, v in d.items()}
        one.update(q=d["q"][rows], starts=ints([0, reqs[b][1]]), tables=d["tables"][b:b + 1], lengths=d["lengths"][b:b + 1],
                   slots=d["slots"][rows], masks=d["masks"][rows].contiguous())
        if gate:
            one["gate"] = d["gate"][rows]
        tree_check(one, want[rows], D, act, cache)


@pytest.mark.parametrize("size", [2.0 ** 99, 2.0 ** 60, 2.0 ** -60, 2.0 ** -100, 0.0])
def test_bf16_queries_of_any_size_over_an_8_bit_cache(size):
    """They are multiplied in fp16, by a power of two of each row that the scores undo."""
    torch = torch_()
    d, n_pages, width = tree_case([(90, 7, 0), (200, 3, 0)], 4, 2, 128, 16, "bf16", "e4m3", 41, False)
    d["q"] = (d["q"].float() * size).to(torch.bfloat16)
    scale = 0.0884 / size if 0 < size < 2.0 ** 90 and size > 2.0 ** -90 else 0.0884 * (2.0 ** -99 if size > 1 else 2.0 ** 99)
    c = lib.PagedCache(4, 2, 128, 16, n_pages, 2, width, dtype="bf16", cache_dtype="e4m3", max_new=7)
    out = c.attend_tree(**d, scale=scale)
    assert c.status() == (0, 0)
    tree_check(d, out, 128, "bf16", "e4m3", scale)


def test_rows_with_strides_and_rows_of_nothing():
    """Queries, gates and outputs as views with other strides; no rows, no requests."""
    torch = torch_()
    d, n_pages, width = tree_case([(300, 9, 0), (64, 4, 0)], 6, 3, 64, 32, "f16", "f16", 51, True)
    c = lib.PagedCache(6, 3, 64, 32, n_pages, 2, width, max_new=9)
    want = c.attend_tree(**d)
    rows = d["q"].shape[0]
    for make in (lambda x: torch.empty(6, rows, 64, dtype=x.dtype, device="cuda").transpose(0, 1),
                 lambda x: torch.empty(rows, 6, 200, dtype=x.dtype, device="cuda")[:, :, 64:128]):
        q, gate, out = (make(d["q"]) for _ in range(3))
        q.copy_(d["q"])
        gate.copy_(d["gate"])
        out.zero_()
        assert torch.equal(c.attend_tree(**{**d, "q": q, "gate": gate}, out=out), want)
    none = ints(np.zeros(0))
    q0 = d["q"][:0]
    e = dict(q=q0, starts=ints([0, 0, 0]), tables=d["tables"], lengths=d["lengths"], k_cache=d["k_cache"], v_cache=d["v_cache"])
    assert c.attend_tree(**e).shape == q0.shape
    assert c.attend_tree(**{**e, "starts": ints([0]), "tables": d["tables"][:0], "lengths": none}).shape == q0.shape
    assert c.status() == (0, 0)


def test_a_gate_that_is_not_finite_concerns_its_element_alone():
    torch = torch_()
    for shape, reqs in ((0, [(300, 9, 0)]), (1, [(6000, 5, 0), (40, 2, 0)])):
        Hq, Hkv, D, page, act, cache, _ = SHAPES[shape]
        d, n_pages, width = tree_case(reqs, Hq, Hkv, D, page, act, cache, 61, True)
        c = lib.PagedCache(Hq, Hkv, D, page, n_pages, len(reqs), width, dtype=act, cache_dtype=cache, max_new=9)
        want = c.attend_tree(**d)
        g = d["gate"].clone()
        flat = g.view(-1)
        flat[5::37], flat[9::41], flat[12::43] = float("nan"), float("inf"), float("-inf")
        got = c.attend_tree(**{**d, "gate": g})
        assert torch.equal(got.isnan(), g.isnan())
        assert (got[g == float("-inf")] == 0).all()
        same = g.isfinite()
        # one reciprocal serves four elements: a neighbour's other divisor moves a value by 2^-21 or less before its
        # rounding, so by one step of the output at most
        a, b = got[same].double(), want[same].double()
        assert ((a - b).abs() <= torch.finfo(got.dtype).eps * b.abs() + 2.0 ** -24).all()
