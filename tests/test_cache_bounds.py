"""Host-side checks that need no GPU: arguments of the paged cache whose offsets or scales pass what the kernels hold."""
import pytest

from tests.test_cache_abi import DENSE, L, P, status  # noqa: F401  (L: the library, a fixture)

LEAST = -(1 << 63)


@pytest.mark.parametrize("change", [
    dict(q_row=LEAST), dict(k_row=LEAST), dict(v_head=LEAST), dict(o_head=LEAST), dict(k_row=-(1 << 40)), dict(k_head=-(1 << 30)),
    dict(q_row=1 << 39, n_rows=1 << 24), dict(k_row=-(1 << 39), n_rows=1 << 24), dict(v_row=(1 << 36) + 8, n_rows=1 << 24),
    dict(o_row=1 << 39, n_rows=(1 << 21) + 1)], ids=str)
def test_write_refuses_rows_whose_offsets_pass_63_bits(L, change):  # noqa: F811
    assert status(L, write=change) == -1


def test_write_takes_rows_as_far_apart_as_they_may_be(L):  # noqa: F811
    assert status(L, write=dict(q_row=1 << 36, k_row=-(1 << 36), v_head=(1 << 30) - 8, n_rows=1 << 24)) == 0
    assert status(L, write=dict(q_row=(1 << 40) - 8, n_rows=1 << 20)) == 0


@pytest.mark.parametrize("change", [dict(q_row=LEAST), dict(g_head=LEAST), dict(o_row=LEAST), dict(q_row=-(1 << 40))], ids=str)
def test_attend_refuses_rows_whose_offsets_pass_63_bits(L, change):  # noqa: F811
    assert status(L, attend=change) == -1


def test_pages_whose_offsets_pass_63_bits(L):  # noqa: F811
    far = 1 << 37
    for n_pages, page, want in ((64, far, 0), (1 << 23, far, 0), ((1 << 23) + 1, far, -1), ((1 << 27) - 1, far, -1),
                                ((1 << 27) - 1, 1 << 33, 0), ((1 << 27) - 1, DENSE, 0), (1, -far, -1), (1, LEAST, -1)):
        cfg = dict(n_pages=n_pages)
        for change in (dict(k_page=page), dict(v_page=page)):
            assert status(L, cfg=cfg, write=change) == want and status(L, cfg=cfg, attend=change) == want, (n_pages, page)


@pytest.mark.parametrize("scale", [1e39, -1e39, 3.4e38, -2.5e38, 1e300])
def test_attend_refuses_scales_that_fp32_does_not_hold(L, scale):  # noqa: F811
    """The kernels multiply scores by scale * log2(e) in fp32: past 2.35e38 that is an infinity, and the outputs NaN."""
    assert status(L, attend=dict(scale=scale)) == -1


@pytest.mark.parametrize("scale", [0.0, -0.0625, 1e-300, 1e30, 2.3e38, -2.3e38])
def test_attend_takes_every_other_scale(L, scale):  # noqa: F811
    assert status(L, attend=dict(scale=scale)) == 0
