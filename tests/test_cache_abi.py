"""Host-side checks of the paged cache's entry points that need no GPU: the shapes and arguments that are refused, with
the documented status, before any device is touched; and the float64 oracle against closed forms."""
import ctypes

import numpy as np
import pytest

import oracle.cache_oracle as O
from w4a16_top_mixture_gb300 import build, lib

OK = dict(n_heads=16, n_kv_heads=2, head_dim=256, page_size=16, n_pages=64, max_requests=8, max_pages=32, act_dtype=0,
          cache_dtype=0, rope_dim=64, rope_theta=1e7, gamma_offset=1.0, norm_eps=1e-6)
P = 4096                                             # an aligned address that nothing reads
DENSE = 2 * 16 * 256
PLAN = dict(lengths=P, new_tokens=P, tables=P, table_stride=32, free_pages=P, free_state=P, free_state_out=P, lengths_out=P,
            starts=P, slots=P, positions=P, n_requests=4, n_rows=4)
WRITE = dict(q=P, q_row=4096, q_head=256, k=P, k_row=4096, k_head=256, v=P, v_row=4096, v_head=256, o=P, o_row=4096, o_head=256,
             q_gamma=P, k_gamma=P, positions=P, slots=P, k_cache=P, v_cache=P, k_page=DENSE, v_page=DENSE, k_scale=0, v_scale=0,
             n_rows=4)
ATTEND = dict(q=P, q_row=4096, q_head=256, gate=P, g_row=4096, g_head=256, out=P, o_row=4096, o_head=256, tables=P,
              table_stride=32, lengths=P, k_cache=P, v_cache=P, k_page=DENSE, v_page=DENSE, k_scale=0, v_scale=0, n_requests=8,
              scale=0.0625)


@pytest.fixture(scope="module")
def L():
    build.build()
    return lib.load_library()


def status(L, cfg=(), plan=None, write=None, attend=None):
    c = lib.CacheConfig(*{**OK, **dict(cfg)}.values())
    packed = [f.pack(*{**base, **d}.values()) if d is not None else None
              for f, base, d in ((lib.CACHE_PLAN, PLAN, plan), (lib.CACHE_WRITE, WRITE, write), (lib.CACHE_ATTEND, ATTEND, attend))]
    return L.moe_debug_cache_check(ctypes.byref(c), *packed)


def test_well_formed_calls_pass(L):
    assert status(L, plan={}, write={}, attend={}) == 0
    assert status(L, cfg=dict(act_dtype=1, cache_dtype=2), write=dict(k_scale=P, v_scale=P), attend=dict(k_scale=P, v_scale=P)) == 0
    assert status(L, plan=dict(new_tokens=0, n_rows=0, slots=0, positions=0)) == 0
    assert status(L, plan=dict(n_requests=0, lengths=0, tables=0, lengths_out=0)) == 0
    assert status(L, write=dict(q=0, o=0, q_gamma=0, k_gamma=0)) == 0
    assert status(L, write=dict(n_rows=0, k=0)) == 0
    assert status(L, attend=dict(gate=0)) == 0
    assert status(L, attend=dict(n_requests=0, q=0)) == 0


@pytest.mark.parametrize("change", [
    dict(n_heads=15), dict(n_heads=0), dict(n_heads=256, n_kv_heads=2), dict(n_kv_heads=0), dict(n_kv_heads=257, n_heads=257),
    dict(head_dim=96), dict(head_dim=0), dict(page_size=8), dict(page_size=24), dict(page_size=512), dict(page_size=0),
    dict(n_pages=0), dict(n_pages=1 << 27), dict(max_pages=0), dict(max_pages=1 << 27), dict(max_requests=0),
    dict(max_requests=4097), dict(max_requests=4096, max_pages=1 << 17), dict(act_dtype=2), dict(act_dtype=1), dict(cache_dtype=3), dict(rope_dim=8), dict(rope_dim=272),
    dict(rope_dim=-16), dict(rope_theta=1.0), dict(rope_theta=float("nan")), dict(norm_eps=-1.0), dict(norm_eps=float("inf")),
    dict(gamma_offset=float("nan"))], ids=str)
def test_shapes_without_a_kernel_are_unsupported(L, change):
    assert status(L, cfg=change) == -2
    h = ctypes.c_void_p()
    c = lib.CacheConfig(*{**OK, **change}.values())
    assert L.moe_cache_create(ctypes.byref(c), ctypes.byref(h)) == -2 and h.value is None


@pytest.mark.parametrize("change", [
    dict(lengths=0), dict(tables=0), dict(tables=P + 2), dict(table_stride=31), dict(free_pages=0), dict(free_state=0),
    dict(free_state_out=0), dict(lengths_out=0), dict(starts=0), dict(slots=0), dict(positions=0), dict(new_tokens=P + 1),
    dict(n_requests=9), dict(n_requests=-1), dict(n_rows=-1), dict(n_rows=1 << 31)], ids=str)
def test_plan_refuses(L, change):
    assert status(L, plan=change) == -1


@pytest.mark.parametrize("change", [
    dict(q=0), dict(o=0), dict(q=P + 8), dict(k=0), dict(v=P + 2), dict(q_row=4100), dict(k_head=4), dict(v_row=1 << 40), dict(k_head=1 << 30),
    dict(q_gamma=P + 8), dict(k_gamma=P + 2), dict(positions=0), dict(slots=P + 1), dict(k_cache=0), dict(v_cache=P + 8),
    dict(k_page=DENSE - 8), dict(v_page=DENSE + 4), dict(k_scale=P), dict(v_scale=P), dict(n_rows=-1),
    dict(n_rows=(1 << 24) + 1)], ids=str)
def test_write_refuses(L, change):
    assert status(L, write=change) == -1


@pytest.mark.parametrize("change", [
    dict(q=0), dict(q=P + 8), dict(gate=P + 2), dict(out=0), dict(out=P + 4), dict(q_row=2), dict(g_head=12), dict(o_row=7),
    dict(tables=0), dict(table_stride=31), dict(lengths=0), dict(lengths=P + 2), dict(k_cache=P + 8), dict(v_cache=0),
    dict(k_page=DENSE - 8), dict(v_page=DENSE + 4), dict(k_scale=P, v_scale=P), dict(n_requests=9), dict(n_requests=-1),
    dict(scale=float("nan")), dict(scale=float("inf"))], ids=str)
def test_attend_refuses(L, change):
    assert status(L, attend=change) == -1


def test_an_8_bit_cache_needs_its_scales_and_whole_16_byte_pages(L):
    cfg, both = dict(cache_dtype=2), dict(k_scale=P, v_scale=P)
    assert status(L, cfg=cfg, write={}) == -1 and status(L, cfg=cfg, attend={}) == -1
    assert status(L, cfg=cfg, write=dict(k_scale=P)) == -1 and status(L, cfg=cfg, attend=dict(v_scale=P)) == -1
    assert status(L, cfg=cfg, attend=dict(both, k_page=DENSE + 8)) == -1


def test_pages_are_whole_lines_apart(L):
    narrow = dict(cache_dtype=2, head_dim=64, rope_dim=64)
    both = dict(k_scale=P, v_scale=P)
    for change, want in ((dict(), 0), (dict(k_page=DENSE + 128), 0), (dict(v_page=DENSE + 64), -1), (dict(k_page=DENSE + 192), -1)):
        assert status(L, cfg=narrow, attend=dict(both, **change)) == want, change
        assert status(L, cfg=narrow, write=dict(both, **change)) == want, change


def test_null_handles_and_no_device(L):
    import torch
    h = ctypes.c_void_p()
    c = lib.CacheConfig(*OK.values())
    assert L.moe_cache_create(None, ctypes.byref(h)) == -1 and L.moe_cache_create(ctypes.byref(c), None) == -1
    assert L.moe_debug_cache_check(None, None, None, None) == -1
    for f in (L.moe_cache_plan, L.moe_cache_write, L.moe_cache_attend):
        assert f(None, None, None) == -1
    assert L.moe_cache_get_status(None, None) == -1
    L.moe_cache_destroy(None)
    if not torch.cuda.is_available():
        assert L.moe_cache_create(ctypes.byref(c), ctypes.byref(h)) == -6 and h.value is None


# ---- the oracle ----

def test_oracle_attention_closed_forms():
    rng = np.random.default_rng(0)
    k, v = rng.normal(size=(3, 1, 16, 64)), rng.normal(size=(3, 1, 16, 64))
    tables = np.array([[2, 0], [1, 7]])
    q = np.zeros((2, 2, 64))
    out, _, _ = O.attend(q, tables, [20, 1], k, v, 0.125)          # a zero query: the mean of the values
    np.testing.assert_allclose(out[0, 1], np.concatenate([v[2, 0], v[0, 0, :4]]).mean(0))
    np.testing.assert_allclose(out[1, 0], v[1, 0, 0])
    q[0, 0] = 1e4 * k[0, 0, 3]                                      # a query far along one key: its value
    k[0, 0, 3] *= 4
    out, _, _ = O.attend(q, tables, [20, 0], k, v, 0.125)
    np.testing.assert_allclose(out[0, 0], v[0, 0, 3])
    assert (out[1] == 0).all()
    gated, _, _ = O.attend(q, tables, [20, 0], k, v, 0.125, gate=np.zeros_like(q))
    np.testing.assert_allclose(gated, out / 2)


def test_oracle_rotation_and_norm():
    rng = np.random.default_rng(1)
    x = rng.normal(size=(2, 3, 64))
    y, _ = O.norm_rope(x, np.zeros(64), np.array([0, 5]), 32, 1e4, 1.0, 0.0)
    np.testing.assert_allclose((y * y).mean(-1), 1.0)               # a rotation keeps the norm
    np.testing.assert_allclose(y[0], x[0] / np.sqrt((x[0] ** 2).mean(-1, keepdims=True)))
    a, _ = O.norm_rope(x, None, np.array([7, 9]), 64, 1e4, 0.0, 0.0)
    b, _ = O.norm_rope(x, None, np.array([107, 109]), 64, 1e4, 0.0, 0.0)
    np.testing.assert_allclose((a[0] * a[1]).sum(-1), (b[0] * b[1]).sum(-1))   # products see distances alone


def test_oracle_plan_by_hand():
    tables = np.full((3, 4), -1, np.int32)
    tables[0, :2], tables[1, :1] = (5, 6), (7,)
    s, p, st, ln, fs, tb, ring = O.plan([32, 16, 0], [1, -1, 17], tables, [9, 8, 4, 3, 2, 1, 0, 0, 0, 0], [1, 3, 0], 20, 16, 10)
    assert list(s) == [8 * 16] + [4 * 16 + i for i in range(16)] + [3 * 16] + [-1, -1]
    assert list(p) == [32] + list(range(17)) + [0, 0] and list(st) == [0, 1, 1, 18] and list(ln) == [33, 0, 17]
    assert list(fs) == [4, 1, 0] and list(tb[2]) == [4, 3, -1, -1] and tb[0, 2] == 8 and ring[4] == 7
