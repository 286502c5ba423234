"""What lib.PagedCache hands to the library, without a GPU: a handle whose library only records the calls."""
import types

import pytest

from w4a16_top_mixture_gb300 import lib


@pytest.fixture
def cache():
    import torch
    calls = []
    take = lambda f: lambda h, args, stream: calls.append((f, args)) or 0  # noqa: E731
    c = object.__new__(lib.PagedCache)
    c.__dict__.update(lib=types.SimpleNamespace(moe_cache_write=take("write"), moe_cache_attend=take("attend"), moe_cache_plan=take("plan")),
                      h=None, dtype=torch.float16, cache_dtype=torch.float16, n_heads=4, n_kv_heads=2, head_dim=64, page_size=16, n_pages=6,
                      max_pages=3, pool_shape=(6, 2, 16, 64), device=torch.device("cpu"), _torch=torch, _dev=-1, _i32=torch.int32,
                      _f32=torch.float32, _raw_stream=lambda dev: 0, calls=calls)
    return c


def inputs(rows=3):
    import torch
    i32 = lambda *s: torch.zeros(*s, dtype=torch.int32)  # noqa: E731
    rand = lambda *s: torch.zeros(*s, dtype=torch.float16)  # noqa: E731
    pool = rand(6, 2, 2, 16, 64)
    return types.SimpleNamespace(q=rand(rows, 4, 64), k=rand(rows, 2, 64), v=rand(rows, 2, 64), positions=i32(rows), slots=i32(rows),
                                 kc=pool[:, 0], vc=pool[:, 1], tables=i32(rows, 3), lengths=i32(rows))


def test_pools_are_handed_over_with_their_own_strides(cache):
    x = inputs()
    cache.attend(x.q, x.tables, x.lengths, x.kc, x.vc.contiguous())
    args = lib.CACHE_ATTEND.unpack(cache.calls[0][1])
    assert args[12] == x.kc.data_ptr() and args[14:16] == (2 * 2 * 16 * 64, 2 * 16 * 64)


def test_pools_whose_pages_overlap_are_refused(cache):
    """One page shown as six, or pages closer than they are long: with dense strides the kernels would leave the tensor."""
    x = inputs()
    one = x.kc[:1].expand(6, 2, 16, 64)
    near = x.kc.new_zeros(6 * 2 * 16 * 64).as_strided((6, 2, 16, 64), (1024, 1024, 64, 1))
    for bad in (one, near):
        for kc, vc in ((bad, x.vc), (x.kc, bad)):
            with pytest.raises(ValueError):
                cache.attend(x.q, x.tables, x.lengths, kc, vc)
            with pytest.raises(ValueError):
                cache.write(x.q, x.k, x.v, x.positions, x.slots, kc, vc)
    assert not cache.calls


def test_a_pool_of_one_page_may_have_any_page_stride(cache):
    cache.n_pages, cache.pool_shape = 1, (1, 2, 16, 64)
    x = inputs()
    for stride in (0, 5, 12345):
        one = x.kc[:1].as_strided((1, 2, 16, 64), (stride, 1024, 64, 1))
        cache.attend(x.q, x.tables, x.lengths, one, one)
        assert lib.CACHE_ATTEND.unpack(cache.calls.pop()[1])[14:16] == (2 * 16 * 64,) * 2


def test_an_output_without_queries_is_refused(cache):
    """It came back as the result of the call, unwritten."""
    x = inputs()
    with pytest.raises(ValueError):
        cache.write(None, x.k, x.v, x.positions, x.slots, x.kc, x.vc, q_out=x.q)
    assert not cache.calls
    assert cache.write(None, x.k, x.v, x.positions, x.slots, x.kc, x.vc) is None and len(cache.calls) == 1
