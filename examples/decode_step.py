"""A decode step of a small hybrid decoder over the paged key-value cache: for every layer, gated attention (projections in
torch, norm, rotary embedding, cache and attention in the library) and the routed MoE block, each with its residual.

  python examples/decode_step.py [--layers 2] [--requests 8] [--steps 32] [--tiny] [--cache e4m3]

One plan serves the step's layers: the page plan, the write and the attention share one handle, and every layer has pools
of its own. The whole step is captured once as a CUDA graph and replayed; lengths, tables and the ring of free pages are
updated in place on the GPU."""
import argparse
import os
import sys
import time

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from w4a16_top_mixture_gb300 import lib, synth  # noqa: E402

EPS, THETA = 1e-6, 1e7


def rms_norm(x, gamma):
    x = x.float()
    return (x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS) * gamma.float()).half()


class Layer:
    """One decoder layer: the attention's weights and pools, and the MoE block. q and its gate lie side by side per head,
    then k, then v, in one projection."""

    def __init__(self, cfg, heads, kv_heads, dim, rows, pool_shape, pool_dtype, seed):
        gen = torch.Generator(device="cuda")
        gen.manual_seed(seed)
        rand = lambda *s, gain=1.0: (torch.randn(*s, generator=gen, device="cuda") * gain).half()  # noqa: E731
        H = cfg.hidden
        self.heads, self.kv_heads, self.dim = heads, kv_heads, dim
        self.w_in = rand(H, (2 * heads + 2 * kv_heads) * dim, gain=H ** -0.5)
        self.w_out = rand(heads * dim, H, gain=(heads * dim) ** -0.5)
        self.gamma = rand(H, gain=0.05) + 1
        self.q_gamma, self.k_gamma = rand(dim, gain=0.05), rand(dim, gain=0.05)
        self.k_pool = torch.zeros(pool_shape, dtype=pool_dtype, device="cuda")
        self.v_pool = torch.zeros(pool_shape, dtype=pool_dtype, device="cuda")
        self.scales = {}
        if pool_dtype == torch.float8_e4m3fn:
            self.scales = dict(k_scale=torch.full((kv_heads,), 0.03, device="cuda"), v_scale=torch.full((kv_heads,), 0.03, device="cuda"))
        self.moe = lib.MoeBlock.from_config(cfg, max_tokens=rows)
        self.moe.load_weights(lib.upload_weights(synth.gen_layer(cfg, seed, with_gamma=True)))

    def project(self, h):
        x = (rms_norm(h, self.gamma) @ self.w_in).view(h.shape[0], 2 * self.heads + 2 * self.kv_heads, self.dim)
        qg = x[:, :2 * self.heads].view(h.shape[0], self.heads, 2, self.dim)
        k, v = x[:, 2 * self.heads:].split(self.kv_heads, 1)
        return qg[:, :, 0], qg[:, :, 1], k, v

    def __call__(self, h, cache, plan, tables):
        q, gate, k, v = self.project(h)
        q = cache.write(q, k, v, plan.positions, plan.slots, self.k_pool, self.v_pool, q_gamma=self.q_gamma, k_gamma=self.k_gamma,
                        **self.scales)
        y = cache.attend(q, tables, plan.lengths, self.k_pool, self.v_pool, gate=gate, **self.scales)
        return self.moe.forward_residual(h + y.view(h.shape[0], -1) @ self.w_out, eps=EPS)


class Decoder:
    """Layers over one cache, and the step's state on the GPU: lengths, tables, the ring of free pages."""

    def __init__(self, cfg, layers, requests, heads, kv_heads, dim, page=16, max_tokens=1024, cache_dtype="f16", rope=None, seed=1):
        max_pages = -(-max_tokens // page)
        n_pages = requests * max_pages
        self.cache = lib.PagedCache(heads, kv_heads, dim, page, n_pages, requests, max_pages, cache_dtype=cache_dtype,
                                    rope_dim=dim // 4 if rope is None else rope, rope_theta=THETA, gamma_offset=1.0, eps=EPS)
        self.layers = [Layer(cfg, heads, kv_heads, dim, requests, self.cache.pool_shape, self.cache.cache_dtype, seed + i)
                       for i in range(layers)]
        i32 = lambda *s: torch.zeros(*s, dtype=torch.int32, device="cuda")  # noqa: E731
        self.tables, self.ring = i32(requests, max_pages), torch.arange(n_pages, dtype=torch.int32, device="cuda")
        self.plan = lib.CachePlan(i32(requests), i32(requests), i32(requests + 1), i32(requests),
                                  torch.tensor([0, n_pages, 0], dtype=torch.int32, device="cuda"))

    def step(self, h):
        """One token of every request: h [requests, hidden] fp16 -> the last layer's hidden states."""
        p = self.plan
        self.cache.plan(p.lengths, None, self.tables, self.ring, p.free_state, h.shape[0], out=p)
        for layer in self.layers:
            h = layer(h, self.cache, p, self.tables)
        return h

    def check(self):
        for what in (self.cache, *(layer.moe for layer in self.layers)):
            status, flags = what.status()
            if status:
                raise lib.MoeError(status, f"flags {flags}")


def main():
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--layers", type=int, default=2)
    ap.add_argument("--requests", type=int, default=8)
    ap.add_argument("--steps", type=int, default=32)
    ap.add_argument("--tiny", action="store_true")
    ap.add_argument("--cache", default="f16", choices=("f16", "e4m3"))
    a = ap.parse_args()
    cfg = synth.TINY if a.tiny else synth.PROD
    heads, kv_heads, dim = (4, 2, 64) if a.tiny else (16, 2, 256)
    d = Decoder(cfg, a.layers, a.requests, heads, kv_heads, dim, max_tokens=a.steps + 16, cache_dtype=a.cache)
    h = torch.randn(a.requests, cfg.hidden, device="cuda", dtype=torch.float16)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        d.step(h)                                   # warm-up: library handles of torch
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = d.step(h)
    torch.cuda.synchronize()
    t = time.perf_counter()
    for _ in range(a.steps):
        graph.replay()
        h.copy_(rms_norm(out, torch.ones_like(out[0])))
    torch.cuda.synchronize()
    t = time.perf_counter() - t
    d.check()
    print(f"{a.layers} layers, {a.requests} requests, {a.steps} steps: {t / a.steps * 1e6:.0f} us per step, "
          f"{a.requests * a.steps / t:.0f} tokens/s, lengths {d.plan.lengths.tolist()[:4]}..., finite {bool(torch.isfinite(out).all())}")


if __name__ == "__main__":
    main()
