"""What the paged cache's handle reports and when: calls in graphs on streams that it never sees, captures."""
import numpy as np
import pytest

from tests.test_gpu_cache import attend_case, attend_check, run_plan, torch_
from w4a16_top_mixture_gb300 import build, lib

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    build.build()
    lib.load_library()


def test_status_waits_for_a_graph_on_another_stream():
    """A captured call, replayed behind 50 ms of other work on a stream of its own: its report is there when status()
    returns, and what it computes is not disturbed."""
    torch = torch_()
    d, n_pages, width = attend_case([9000, 40, 3000], 16, 2, 256, 16, "f16", "f16", 21)
    d["tables"][0, 0] = n_pages                               # reads as zeros, and is reported
    c = lib.PagedCache(16, 2, 256, 16, n_pages, 3, width)
    want = c.attend(**d)
    assert c.status() == (-1, 4)
    attend_check(d, want, 16, 2, 256, "f16", "f16")
    out = torch.zeros_like(want)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        c.attend(**d, out=out)
    side = torch.cuda.Stream()
    for _ in range(3):
        out.zero_()
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            torch.cuda._sleep(100_000_000)
            g.replay()
        assert c.status() == (-1, 4) and c.status() == (0, 0)
        assert torch.equal(out, want)


def test_status_is_refused_in_a_capture():
    torch = torch_()
    d, n_pages, width = attend_case([300], 16, 2, 256, 16, "f16", "f16", 22)
    c = lib.PagedCache(16, 2, 256, 16, n_pages, 1, width)
    want = c.attend(**d)
    out = torch.empty_like(want)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        with pytest.raises(RuntimeError):
            c.status()
        c.attend(**d, out=out)
    g.replay()
    assert c.status() == (0, 0) and torch.equal(out, want)


def test_plan_drops_pages_that_the_ring_has_no_room_for():
    """Two ended requests hold the same pages: the ring takes what it has room for and reports the rest; the entries that
    are free already stay, and a request of the same call takes the first of them."""
    c = lib.PagedCache(1, 1, 64, 16, 8, 4, 2)
    ring = [6, 7, -1, -1, -1, 2, 3, 4]                        # from entry 5 on: pages 2, 3, 4, 6, 7
    for in_place in (False, True):
        got = run_plan(c, [32, 32, 16], [-1, -1, 1], [[0, 1], [0, 1], [5, -1]], ring, [5, 5, 0], 1, in_place)
        slots, positions, starts, lengths, state, tables, out = (x.tolist() for x in got)
        assert slots == [2 * 16] and positions == [16] and lengths == [0, 0, 17] and tables[2] == [5, 2]
        assert out == [6, 7, 0, 1, 0, 2, 3, 4] and state == [6, 5 - 1 + 3, 0]
        assert c.status() == (-1, 8) and c.status() == (0, 0)
    # with room for all of them nothing is reported: a page in two places is the caller's to find
    got = run_plan(c, [32, 32], [-1, -1], [[0, 1], [0, 1]], ring, [5, 4, 0], 0)
    assert got[6].tolist() == [6, 0, 1, 0, 1, 2, 3, 4] and got[4].tolist() == [5, 8, 0] and c.status() == (0, 0)


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("B", [60, 1025, 4096])
def test_plan_of_many_requests_with_pages_in_common(B, in_place):
    """Every third request ends with the pages of all others, in a ring that is nearly full, while the rest take pages."""
    page, n_pages, width, room = 16, 20000, 40, 333
    count, head = n_pages - room, 19000
    rng = np.random.default_rng(B)
    free = rng.permutation(n_pages)[:count]
    ring = np.full(n_pages, -9)
    ring[(head + np.arange(count)) % n_pages] = free
    ends = np.arange(B) % 3 == 0
    tables = np.full((B, width), -7)
    tables[:, :30] = np.arange(30)
    lengths = np.where(ends, 480, 32)
    c = lib.PagedCache(1, 1, 64, page, n_pages, B, width)
    got = run_plan(c, lengths, np.where(ends, -1, 32), tables, ring, [head, count, 0], 32 * B, in_place)
    slots, positions, starts, out_len, state, out_tables, out = got
    n = int((~ends).sum())
    assert c.status() == (-1, 8)
    assert state.tolist() == [(head + 2 * n) % n_pages, count - 2 * n + room, 0]
    assert (out_len == np.where(ends, 0, 64)).all()
    assert (out_tables[~ends][:, 2:4] == free[:2 * n].reshape(-1, 2)).all()
    want = ring.copy()
    want[(head + count + np.arange(room)) % n_pages] = (np.arange(room) % 30)
    assert (out == want).all()
