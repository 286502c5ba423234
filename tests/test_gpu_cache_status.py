"""What the paged cache's handle reports and when: calls in graphs on streams that it never sees, captures."""
import pytest

from tests.test_gpu_cache import attend_case, attend_check, torch_
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
