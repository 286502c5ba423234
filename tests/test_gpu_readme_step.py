"""The step of several new tokens as README.md shows it, run as a loop over requests that fork: what the calls hand out and take
back stays consistent."""
import os
import re

import numpy as np
import pytest

from test_gpu_cache import gen_of, ints, randn, torch_
from test_gpu_tree import random_parents
from w4a16_top_mixture_gb300 import build, lib

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module", autouse=True)
def _lib():
    build.build()
    lib.load_library()


def shown_step():
    """The lines of README.md's step, from the plan on."""
    text = open(os.path.join(ROOT, "README.md")).read()
    block = next(b for b in re.findall(r"```python\n(.*?)```", text, re.S) if "cache.fork(" in b)
    lines = block.splitlines()
    return "\n".join(lines[next(i for i, line in enumerate(lines) if line.startswith("p = cache.plan")):])


def test_the_step_of_the_readme_holds_over_forks():
    torch = torch_()
    B, Hq, Hkv, D, page, n_pages, width, new = 6, 4, 2, 64, 16, 200, 20, 24
    rng, gen = np.random.default_rng(1), gen_of(1)
    cache = lib.PagedCache(n_heads=Hq, n_kv_heads=Hkv, head_dim=D, page_size=page, n_pages=n_pages, max_requests=B, max_pages=width,
                           max_new=64)
    k0, v0 = (torch.zeros(cache.pool_shape, device="cuda", dtype=torch.float16) for _ in range(2))
    names = dict(cache=cache, k0=k0, v0=v0, pools=cache.pools([k0, v0]), lengths=ints(np.zeros(B)), free_state=ints([0, n_pages, 0]),
                 tables=torch.full((B, width), -1, dtype=torch.int32, device="cuda"), n_rows=B * new,
                 free_pages=torch.arange(n_pages, dtype=torch.int32, device="cuda"), refs=ints(np.zeros(n_pages)))
    step = compile(shown_step(), "README.md", "exec")
    alive = np.array([True, True, False, False, False, False])
    # which requests end at a step, and who forks whom after it
    for end, fork in (([], [(0, 2), (1, 3)]), ([], [(0, 4)]), ([0], [(4, 5)]), ([3, 4], []), ([], [(2, 0)]), ([2, 5], [])):
        n = np.where(alive, new, 0)
        parents = np.full(B * new, -1, np.int32)
        parents[:n.sum()] = random_parents(rng, n, "chain")
        counts = np.where(alive, rng.integers(1, new + 1, B), 0)
        counts[end] = -1
        path = np.tile(np.arange(new), (B, 1))
        x = randn(gen, (B * new, Hq + 2 * Hkv, D), "f16")
        src, dst = ([a for a, _ in fork] or [-1]), ([b for _, b in fork] or [0])
        names.update(new_tokens=ints(n), parents=ints(parents), q=x[:, :Hq], k=x[:, Hq:Hq + Hkv], v=x[:, Hq + Hkv:], counts=ints(counts),
                     path=ints(path), src=ints(src), dst=ints(dst))
        exec(step, names)
        f = names["f"]
        names.update(lengths=f.lengths, free_state=f.free_state)
        assert cache.status() == (0, 0)
        alive[end] = False
        alive[[b for _, b in fork]] = True
        ln, tables, (head, count, none) = f.lengths.tolist(), names["tables"].cpu().numpy(), f.free_state.tolist()
        assert none == 0 and all((ln[b] > 0) == alive[b] for b in range(B))
        held = [int(t) for b in range(B) for t in tables[b, :-(-ln[b] // page)]]
        free = [int(names["free_pages"][(head + i) % n_pages]) for i in range(count)]
        assert len(set(free)) == count and not set(free) & set(held)
        assert len(set(held)) + count == n_pages
        np.testing.assert_array_equal(names["refs"].cpu().numpy()[held], [held.count(p) - 1 for p in held])
