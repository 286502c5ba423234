"""The decode example: page plan, cache write, attention and MoE block in one step, eager and as a captured graph. The
attention of its first layer is checked against the float64 oracle over the whole history of every request."""
import importlib.util
import os

import numpy as np
import pytest

import oracle.cache_oracle as O
from w4a16_top_mixture_gb300 import build, synth

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def example():
    build.build()
    spec = importlib.util.spec_from_file_location("decode_step", os.path.join(ROOT, "examples", "decode_step.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def f64(t):
    return t.detach().cpu().double().numpy()


@pytest.mark.parametrize("cache", ["f16", "e4m3"])
def test_steps_match_the_oracle(example, cache):
    import torch
    B, heads, kv_heads, dim, rope, steps = 3, 4, 2, 64, 32, 37
    d = example.Decoder(synth.TINY, 2, B, heads, kv_heads, dim, max_tokens=48, cache_dtype=cache, rope=rope, seed=3)
    layer, seen, outs = d.layers[0], [], []
    project, attend = layer.project, d.cache.attend
    layer.project = lambda h: seen.append([x.clone() for x in project(h)]) or tuple(seen[-1])
    d.cache.attend = lambda *a, **k: outs.append(attend(*a, **k)) or outs[-1]
    gen = torch.Generator(device="cuda")
    gen.manual_seed(5)
    h = torch.randn(B, synth.TINY.hidden, generator=gen, device="cuda").half()
    for _ in range(steps):
        h = d.step(h)
        h = example.rms_norm(h, torch.ones_like(h[0]))
    torch.cuda.synchronize()
    d.check()
    assert d.plan.lengths.tolist() == [steps] * B and torch.isfinite(h).all()
    pos = np.arange(steps)
    qg, kg = f64(layer.q_gamma), f64(layer.k_gamma)
    y = f64(outs[-2])                                   # the last step's two layers: the first's output
    u, uk = 2.0 ** -11, (2.0 ** -4 if cache == "e4m3" else 2.0 ** -11)
    for b in range(B):
        k, _ = O.norm_rope(np.stack([f64(s[2][b]) for s in seen]), kg, pos, rope, example.THETA, 1.0, example.EPS)
        v = np.stack([f64(s[3][b]) for s in seen])
        q, _ = O.norm_rope(f64(seen[-1][0][b])[None], qg, pos[-1:], rope, example.THETA, 1.0, example.EPS)
        pool = lambda x: x.transpose(1, 0, 2)[None]  # noqa: E731  one page that holds every token
        want, size, mag = O.attend(q, np.zeros((1, 1), int), [steps], pool(k), pool(v), dim ** -0.5, f64(seen[-1][1][b])[None])
        # keys and values are rounded to the cache's type (an e4m3 code at least 2^-10 of its scale), q to fp16: a score is
        # off by (u + uk) sum |q k| scale and the code's smallest step
        small = 0.03 * 2.0 ** -10 if cache == "e4m3" else 0.0
        delta = (u + uk) * mag + small * np.abs(q).sum(-1, keepdims=True) * dim ** -0.5 + dim * 2.0 ** -23 * mag
        tol = u * np.abs(want) + size * (np.expm1(2 * delta) + uk + u + 2.0 ** -17) + small + 2.0 ** -24
        assert (np.abs(y[b] - want[0]) <= tol[0]).all()


def test_a_captured_step_repeats_the_eager_one(example):
    import torch
    outs = []
    for captured in (False, True):
        d = example.Decoder(synth.TINY, 2, 5, 4, 2, 64, max_tokens=64, seed=7)
        h = torch.full((5, synth.TINY.hidden), 0.5, device="cuda", dtype=torch.float16)
        h[1:] *= torch.arange(1, 5, device="cuda").half()[:, None]
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            d.step(h)
        torch.cuda.current_stream().wait_stream(side)
        if captured:
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g):
                out = d.step(h)
        for _ in range(20):
            if captured:
                g.replay()
            else:
                out = d.step(h)
            h.copy_(example.rms_norm(out, torch.ones_like(out[0])))
        torch.cuda.synchronize()
        d.check()
        assert d.plan.lengths.tolist() == [21] * 5
        outs.append(out.clone())
    assert torch.equal(*outs)
