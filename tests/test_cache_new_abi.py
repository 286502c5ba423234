"""Host-side checks, without a GPU, of the cache's calls for several new tokens of a request: what is refused, with which
status, before any device is touched; what lib.PagedCache hands over; and the float64 oracle against hand-worked cases."""
import ctypes
import time
import types

import numpy as np
import pytest

import oracle.cache_oracle as O
from test_cache_abi import DENSE, OK, P
from w4a16_top_mixture_gb300 import build, lib

TREE = dict(parents=P, starts=P, lengths=P, slots=P, masks=P, positions=P, n_requests=4, n_rows=9, mask_words=1)
ATTEND = dict(q=P, q_row=4096, q_head=256, gate=P, g_row=4096, g_head=256, out=P, o_row=4096, o_head=256, starts=P, slots=P, masks=P,
              tables=P, table_stride=32, lengths=P, k_cache=P, v_cache=P, k_page=DENSE, v_page=DENSE, k_scale=0, v_scale=0,
              n_requests=8, n_rows=40, mask_words=1, scale=0.0625)
KEEP = dict(counts=P, lengths=P, starts=P, slots=P, path=P, path_stride=8, tables=P, table_stride=32, free_pages=P, free_state=P,
            free_state_out=P, lengths_out=P, refs=P, pools=0, strides=0, n_pools=0, n_requests=8, n_rows=40)
FORK = dict(src=P, dst=P, lengths=P, lengths_out=P, tables=P, table_stride=32, free_pages=P, free_state=P, free_state_out=P, refs=P,
            pools=0, strides=0, n_pools=0, n_entries=3, n_requests=8)


@pytest.fixture(scope="module")
def L():
    build.build()
    return lib.load_library()


def status(L, cfg=(), max_new=64, tree=None, attend=None, keep=None, fork=None):
    c = lib.CacheConfig(*{**OK, **dict(cfg)}.values())
    packed = [f.pack(*{**base, **d}.values()) if d is not None else None
              for f, base, d in ((lib.CACHE_TREE, TREE, tree), (lib.CACHE_ATTEND_TREE, ATTEND, attend), (lib.CACHE_KEEP, KEEP, keep),
                                 (lib.CACHE_FORK, FORK, fork))]
    return L.moe_debug_cache_check_new(ctypes.byref(c), max_new, *packed)


def test_well_formed_calls_pass(L):
    assert status(L, tree={}, attend={}, keep={}, fork={}) == 0
    assert status(L, tree=dict(slots=0), attend=dict(slots=0, masks=0, mask_words=0, gate=0), keep=dict(slots=0, path=0, path_stride=0, refs=0)) == 0
    assert status(L, keep=dict(starts=0, slots=0, path=0, n_rows=0)) == 0
    assert status(L, tree=dict(n_rows=0, masks=0, parents=0), attend=dict(n_rows=0, q=0), keep=dict(n_requests=0, counts=0, lengths=0, tables=0),
                  fork=dict(n_entries=0, src=0, dst=0)) == 0
    assert status(L, attend=dict(n_requests=0, q=0), fork=dict(n_entries=0, n_requests=0, lengths=0, tables=0)) == 0
    for n in (1, 256):
        assert status(L, max_new=n, tree=dict(mask_words=4)) == 0
    assert status(L, cfg=dict(cache_dtype=2), attend=dict(k_scale=P, v_scale=P)) == 0


@pytest.mark.parametrize("max_new", [0, -1, 257])
def test_the_number_of_new_tokens_is_bounded(L, max_new):
    assert status(L, max_new=max_new) == -2


@pytest.mark.parametrize("change", [dict(parents=0), dict(starts=0), dict(lengths=P + 2), dict(slots=P + 1), dict(masks=0), dict(masks=P + 4),
                                    dict(positions=0), dict(n_requests=9), dict(n_requests=-1), dict(n_rows=-1), dict(n_rows=(1 << 24) + 1),
                                    dict(mask_words=0), dict(mask_words=5)], ids=str)
def test_tree_refuses(L, change):
    assert status(L, tree=change) == -1


@pytest.mark.parametrize("change", [
    dict(q=0), dict(q=P + 8), dict(gate=P + 2), dict(out=0), dict(out=P + 4), dict(q_row=2), dict(g_head=12), dict(o_row=7), dict(starts=0),
    dict(starts=P + 1), dict(slots=P + 2), dict(masks=P + 4), dict(tables=0), dict(table_stride=31), dict(lengths=0), dict(k_cache=P + 8),
    dict(v_cache=0), dict(k_page=DENSE - 8), dict(v_page=DENSE + 4), dict(k_scale=P, v_scale=P), dict(n_requests=9), dict(n_requests=-1),
    dict(n_rows=-1), dict(n_rows=(1 << 24) + 1), dict(mask_words=0), dict(mask_words=5), dict(scale=float("nan")), dict(scale=float("inf"))], ids=str)
def test_attend_tree_refuses(L, change):
    assert status(L, attend=change) == -1


@pytest.mark.parametrize("change", [
    dict(counts=0), dict(lengths=0), dict(lengths_out=P + 2), dict(starts=P + 1), dict(slots=P + 1), dict(path=P + 2), dict(path_stride=0),
    dict(path_stride=1 << 40), dict(starts=0), dict(starts=0, slots=0), dict(starts=0, path=0), dict(tables=0), dict(table_stride=31), dict(free_pages=0),
    dict(free_state=0), dict(free_state_out=0), dict(refs=P + 2), dict(n_pools=-1), dict(n_pools=1025), dict(n_pools=1), dict(n_requests=9),
    dict(n_rows=(1 << 24) + 1)], ids=str)
def test_keep_refuses(L, change):
    assert status(L, keep=change) == -1


@pytest.mark.parametrize("change", [
    dict(src=0), dict(dst=P + 2), dict(lengths=0), dict(lengths_out=0), dict(tables=0), dict(table_stride=31), dict(free_pages=0),
    dict(free_state=0), dict(free_state_out=P + 1), dict(refs=0), dict(n_pools=-1), dict(n_pools=1025), dict(n_pools=2), dict(n_entries=-1),
    dict(n_entries=9), dict(n_requests=9), dict(n_requests=-1)], ids=str)
def test_fork_refuses(L, change):
    assert status(L, fork=change) == -1


def test_pools_are_checked_each(L):
    for bad, want in ((P, 0), (P + 8, -1), (0, -1)):
        pools, strides = (ctypes.c_void_p * 3)(P + 4096, bad, P + 8192), (ctypes.c_int64 * 3)(DENSE, DENSE, DENSE)
        at = dict(pools=ctypes.addressof(pools), strides=ctypes.addressof(strides), n_pools=3)
        assert status(L, keep=at) == want and status(L, fork=at) == want
        strides[2] = DENSE - 64
        assert status(L, keep=at) == -1 and status(L, fork=at) == -1


def test_a_pool_named_twice_is_refused(L):
    for at in ((P, P), (P, P + 16, P), (P + 16, P, P + 32, P)):
        n = len(at)
        pools, strides = (ctypes.c_void_p * n)(*at), (ctypes.c_int64 * n)(*([DENSE] * n))
        a = dict(pools=ctypes.addressof(pools), strides=ctypes.addressof(strides), n_pools=n)
        assert status(L, keep=a) == -1 and status(L, fork=a) == -1


def test_pools_are_told_apart_in_time_that_grows_with_their_number(L):
    """Up to 1024 of them at every keep and fork: a pool named twice is found wherever it stands, and eight times the pools take
    nothing like 64 times as long."""
    c = lib.CacheConfig(*OK.values())
    best = {}
    for n in (128, 1024):
        pools = (ctypes.c_void_p * n)(*(P + 4096 * (i * 7919 % 100003) for i in range(n)))
        strides = (ctypes.c_int64 * n)(*([DENSE] * n))
        a = dict(pools=ctypes.addressof(pools), strides=ctypes.addressof(strides), n_pools=n)
        for i, j in ((0, n - 1), (n // 2, n // 2 + 1), (3, n // 3), (n - 2, n - 1)):
            was, pools[j] = pools[j], pools[i]
            assert status(L, keep=a) == -1 and status(L, fork=a) == -1
            pools[j] = was
        args = lib.CACHE_KEEP.pack(*{**KEEP, **a}.values())
        times = []
        for _ in range(60):
            t = time.perf_counter()
            for _ in range(10):
                assert L.moe_debug_cache_check_new(ctypes.byref(c), 64, None, None, args, None) == 0
            times.append(time.perf_counter() - t)
        best[n] = min(times)
    assert best[1024] < 20 * best[128], best


def test_null_handles(L):
    assert L.moe_cache_reserve(None, 8) == -1
    for f in (L.moe_cache_tree, L.moe_cache_attend_tree, L.moe_cache_keep, L.moe_cache_fork):
        assert f(None, None, None) == -1
    assert L.moe_debug_cache_check_new(None, 8, None, None, None, None) == -1


# ---- the binding ----

@pytest.fixture
def cache():
    import torch
    calls = []
    take = lambda f: lambda h, args, stream: calls.append((f, args)) or 0  # noqa: E731
    c = object.__new__(lib.PagedCache)
    names = ("tree", "attend_tree", "keep", "fork")
    c.__dict__.update(lib=types.SimpleNamespace(**{"moe_cache_" + n: take(n) for n in names}), h=None, dtype=torch.float16,
                      cache_dtype=torch.float16, n_heads=4, n_kv_heads=2, head_dim=64, page_size=16, n_pages=6, max_pages=3,
                      pool_shape=(6, 2, 16, 64), device=torch.device("cpu"), _torch=torch, _dev=-1, _i32=torch.int32, _i64=torch.int64,
                      _f32=torch.float32, _raw_stream=lambda dev: 0, calls=calls, max_new=70)
    return c


def test_the_binding_hands_over_what_it_was_given(cache):
    import torch
    i32 = lambda *s: torch.zeros(*s, dtype=torch.int32)  # noqa: E731
    both = torch.zeros(6, 2, 2, 16, 64, dtype=torch.float16)
    pools = cache.pools([both[:, 0], both[:, 1].contiguous()])
    tables, ring, state, lengths = i32(5, 3), i32(6), i32(3), i32(5)
    counts, path, starts, refs = i32(5), i32(5, 7), i32(6), i32(6)
    r = cache.keep(counts, lengths, tables, ring, state, pools, starts=starts, path=path, refs=refs)
    a = lib.CACHE_KEEP.unpack(cache.calls.pop()[1])
    assert a[:8] == (counts.data_ptr(), lengths.data_ptr(), starts.data_ptr(), 0, path.data_ptr(), 7, tables.data_ptr(), 3)
    assert a[8:13] == (ring.data_ptr(), state.data_ptr(), r.free_state.data_ptr(), r.lengths.data_ptr(), refs.data_ptr())
    assert a[15:] == (2, 5, 1 << 24)
    at = (ctypes.c_void_p * 2).from_address(a[13]), (ctypes.c_int64 * 2).from_address(a[14])
    assert list(at[0]) == [t.data_ptr() for t in pools.tensors] and list(at[1]) == [4096, 2048]
    out = cache.fork(i32(2), i32(2), lengths, tables, ring, state, refs, pools, out=lib.CacheState(lengths, state))
    a = lib.CACHE_FORK.unpack(cache.calls.pop()[1])
    assert a[2:4] == (lengths.data_ptr(),) * 2 and a[7:9] == (state.data_ptr(),) * 2 and a[-3:] == (2, 2, 5) and out.lengths is lengths
    t = cache.tree(i32(9), starts, lengths)
    assert t.masks.shape == (9, 2) and lib.CACHE_TREE.unpack(cache.calls.pop()[1])[6:] == (5, 9, 2)
    q = torch.zeros(9, 4, 64, dtype=torch.float16)
    cache.attend_tree(q, starts, tables, lengths, both[:, 0], both[:, 1], masks=t.masks)
    a = lib.CACHE_ATTEND_TREE.unpack(cache.calls.pop()[1])
    assert a[9:14] == (starts.data_ptr(), 0, t.masks.data_ptr(), tables.data_ptr(), 3) and a[17:19] == (4096, 4096) and a[21:] == (5, 9, 2, 0.125)


def test_the_binding_refuses(cache):
    import torch
    i32 = lambda *s: torch.zeros(*s, dtype=torch.int32)  # noqa: E731
    pool = torch.zeros(6, 2, 16, 64, dtype=torch.float16)
    pools = cache.pools([pool])
    q = torch.zeros(9, 4, 64, dtype=torch.float16)
    ok = (i32(5), i32(5), i32(5, 3), i32(6), i32(3))
    for call in (lambda: cache.keep(*ok, [pool]), lambda: cache.keep(*ok, pools, starts=i32(5)), lambda: cache.keep(*ok, pools, starts=i32(6), path=i32(4, 2)),
                 lambda: cache.keep(*ok, pools, starts=i32(6), path=i32(5, 4)[:, ::2]), lambda: cache.keep(*ok, pools, refs=i32(5)),
                 lambda: cache.keep(*ok[:2], i32(4, 3), *ok[3:], pools), lambda: cache.fork(i32(2), i32(3), *ok[1:], i32(6), pools),
                 lambda: cache.tree(i32(9).long(), i32(6), i32(5)), lambda: cache.tree(i32(9), i32(6), i32(5), words=5),
                 lambda: cache.attend_tree(q, i32(6), ok[2], ok[1], pool, pool, masks=torch.zeros(8, 1, dtype=torch.int64)),
                 lambda: cache.attend_tree(q, i32(6), ok[2], ok[1], pool, pool, masks=torch.zeros(9, dtype=torch.int64)),
                 lambda: cache.attend_tree(q.bfloat16(), i32(6), ok[2], ok[1], pool, pool), lambda: cache.pools([pool[:5]]),
                 lambda: cache.attend_tree(q, i32(6), ok[2], ok[1], pool, pool, slots=i32(8))):
        with pytest.raises(ValueError):
            call()
    assert not cache.calls


# ---- the oracle ----

def test_oracle_tree_by_hand():
    masks, positions = O.tree([-1, 0, 0, 2, -1, 9], [0, 5], [12], [False], 6, 1)
    assert masks[:, 0].tolist() == [1, 0b11, 0b101, 0b1101, 0b10000, 0] and positions.tolist() == [7, 8, 8, 9, 7, 0]


def test_oracle_attention_of_new_tokens():
    rng = np.random.default_rng(0)
    k, v, q = rng.normal(size=(3, 1, 16, 8)), rng.normal(size=(3, 1, 16, 8)), rng.normal(size=(4, 2, 8))
    tables = np.array([[2, 0]])
    chain, *_ = O.attend_tree(q, [0, 3], [False], None, tables, [20], k, v, 0.3)
    for i in range(3):                                              # each row as the one token of a shorter request
        one, *_ = O.attend(q[i:i + 1], tables, [18 + i], k, v, 0.3)
        np.testing.assert_allclose(chain[i], one[0])
    assert np.isnan(chain[3]).all()
    masks = np.array([[1], [2], [5], [0]], np.uint64)               # the second does not see the first
    tree, *_ = O.attend_tree(q, [0, 3], [False], masks, tables, [20], k, v, 0.3)
    np.testing.assert_allclose(tree[0], chain[0])
    keys = np.concatenate([k[2, 0], k[0, 0, :1], k[0, 0, 2:3]])
    vals = np.concatenate([v[2, 0], v[0, 0, :1], v[0, 0, 2:3]])
    s = np.exp(keys @ q[1, 0] * 0.3)
    np.testing.assert_allclose(tree[1, 0], s @ vals / s.sum())


def test_oracle_keep_and_fork_by_hand():
    pool = np.arange(6 * 1 * 2 * 1).reshape(6, 1, 2, 1)             # pages of two tokens
    tables, ring = np.array([[4, 1, 0], [4, 5, -1]]), np.array([2, 3, 9, 9, 9, 9])
    refs = np.array([0, 0, 0, 0, 1, 0])
    # request 0: five tokens, the last three new, of which the second and third stay; request 1 ends
    ln, st, tb, rg, rf, (p,) = O.keep([2, -1], [5, 4], [0, 3, 7], [0, 0], [[1, 2], [0, 0]], tables, ring, [0, 2, 0], refs, [pool], 2, 6)
    assert ln.tolist() == [4, 0] and st.tolist() == [0, 4, 0] and rg.tolist() == [2, 3, 0, 5, 9, 9] and rf.tolist() == [0] * 6
    assert p[1, 0, :, 0].tolist() == [3, 0] and p[4, 0, :, 0].tolist() == [8, 9]
    # back to three tokens: the page that holds the third is request 1's too, and is exchanged
    tables = np.array([[5, 4, 0], [1, 4, -1]])
    ln, st, tb, rg, rf, (p,) = O.keep([3, 4], [5, 4], None, None, None, tables, ring, [0, 2, 0], refs, [pool], 2, 6)
    assert tb.tolist() == [[5, 2, 0], [1, 4, -1]] and rf.tolist() == [0] * 6 and st.tolist() == [1, 2, 0] and rg[2] == 0
    assert p[2, 0, :, 0].tolist() == [8, 5]
    ln, st, tb, rg, rf, (p,) = O.fork([0], [1], np.array([3, 0]), np.array([[5, 4], [-1, -1]]), ring, [1, 1, 0], np.zeros(6, int), [pool], 2, 6)
    assert ln.tolist() == [3, 3] and tb[1].tolist() == [5, 3] and rf.tolist() == [0, 0, 0, 0, 0, 1] and p[3, 0, :, 0].tolist() == [8, 7]
    assert st.tolist() == [2, 0, 0]
