"""A decoder at decode time, built from the library's calls: NF4 linears, residual norms, rotary positions,
a paged (quantised) key-value cache and the attention of one new token over it.

    python examples/decoder.py --layers 36 --batch 1 --context 1024 --kv nf4

builds a 3B-shaped stack with random weights, fills the cache to the given context and reports the time of a
decode step replayed as one CUDA graph.  The step is what a serving loop would run: only the activations
`x`, the lengths and the page table change between replays.
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import nf4_weight_only_gb300 as nf4  # noqa: E402


class Layer:
    """Packed weights and norms of one layer, and its cache."""

    def __init__(self, cfg, generator):
        def packed(n, k):
            w = torch.randn((n, k), generator=generator, device="cuda") * k ** -0.5
            return nf4.quantize(w)

        def norm():
            return (1 + 0.1 * torch.randn(cfg.hidden, generator=generator, device="cuda")).to(torch.bfloat16)

        q_rows, kv_rows = cfg.q_heads * cfg.head_dim, cfg.kv_heads * cfg.head_dim
        self.q, self.k, self.v = packed(q_rows, cfg.hidden), packed(kv_rows, cfg.hidden), packed(kv_rows, cfg.hidden)
        self.o = packed(cfg.hidden, q_rows)
        self.gate, self.up = packed(cfg.inter, cfg.hidden), packed(cfg.inter, cfg.hidden)
        self.down = packed(cfg.hidden, cfg.inter)
        self.norm_in, self.norm_mid = norm(), norm()
        pages = cfg.batch * -(-cfg.max_len // cfg.page_size)
        self.cache = nf4.KVCache.empty(cfg.kv, pages, cfg.kv_heads, cfg.page_size, cfg.head_dim)


class Config:
    def __init__(self, hidden=2048, q_heads=16, kv_heads=2, head_dim=128, inter=11008, layers=36, batch=1, max_len=2048,
                 page_size=64, kv="nf4", theta=1e6, eps=1e-6):
        self.__dict__.update(locals())


class Decoder:
    def __init__(self, cfg: Config, seed: int = 0):
        self.cfg = cfg
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.layers = [Layer(cfg, g) for _ in range(cfg.layers)]
        self.norm_out = torch.ones(cfg.hidden, dtype=torch.bfloat16, device="cuda")
        half = cfg.head_dim // 2
        self.inv_freq = (cfg.theta ** (-torch.arange(half, dtype=torch.float64, device="cuda") / half)).float()
        per_seq = -(-cfg.max_len // cfg.page_size)
        # every sequence owns its pages from the start here; a server hands them out as sequences grow
        self.page_table = torch.arange(cfg.batch * per_seq, dtype=torch.int32, device="cuda").view(cfg.batch, per_seq)
        self.lengths = torch.zeros(cfg.batch, dtype=torch.int32, device="cuda")
        self.workspace = nf4.attention_workspace(self.layers[0].cache, cfg.batch, cfg.q_heads)

        def buffer(*shape):
            return torch.empty((cfg.batch, *shape), dtype=torch.bfloat16, device="cuda")

        self.h, self.delta, self.residual, self.out = (buffer(cfg.hidden) for _ in range(4))
        self.q, self.attn = buffer(cfg.q_heads, cfg.head_dim), buffer(cfg.q_heads, cfg.head_dim)
        self.k, self.v = buffer(cfg.kv_heads, cfg.head_dim), buffer(cfg.kv_heads, cfg.head_dim)
        self.gate, self.up = buffer(cfg.inter), buffer(cfg.inter)

    def step(self, x: torch.Tensor) -> torch.Tensor:
        """One token of every sequence: x bf16 [batch, hidden] -> the last norm's output; lengths grow by one."""
        cfg, flat = self.cfg, (self.cfg.batch, -1)
        position = self.lengths.long()
        page = self.page_table.gather(1, (position // cfg.page_size)[:, None])[:, 0].long()
        slots = page * cfg.page_size + position % cfg.page_size  # the new tokens' places, the same in every layer
        positions = self.lengths.clone()[None]
        self.lengths += 1
        self.residual.copy_(x)
        for i, layer in enumerate(self.layers):
            if i == 0:
                nf4.nf4_rmsnorm(self.residual, layer.norm_in, cfg.eps, y=self.h)
            else:
                nf4.nf4_rmsnorm(self.delta, layer.norm_in, cfg.eps, residual=self.residual,
                                residual_out=self.residual, y=self.h)
            (qc, qs), (kc, ks), (vc, vs) = layer.q, layer.k, layer.v
            nf4.nf4_linear_grouped(self.h, [qc, kc, vc], [qs, ks, vs],
                                   [self.q.view(flat), self.k.view(flat), self.v.view(flat)])
            nf4.nf4_rope(self.q, self.k, positions, self.inv_freq, self.q, self.k)
            nf4.nf4_kv_append(layer.cache, self.k, self.v, slots)
            nf4.nf4_attention_decode(layer.cache, self.q, self.page_table, self.lengths, self.attn, self.workspace)
            nf4.nf4_linear(self.attn.view(flat), *layer.o, self.delta)
            nf4.nf4_rmsnorm(self.delta, layer.norm_mid, cfg.eps, residual=self.residual, residual_out=self.residual,
                            y=self.h)
            nf4.nf4_linear_grouped(self.h, [layer.gate[0], layer.up[0]], [layer.gate[1], layer.up[1]],
                                   [self.gate, self.up])
            nf4.nf4_linear(torch.nn.functional.silu(self.gate) * self.up, *layer.down, self.delta)
        nf4.nf4_rmsnorm(self.delta, self.norm_out, cfg.eps, residual=self.residual, residual_out=self.residual,
                        y=self.out)
        return self.out


def main():
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--layers", type=int, default=36)
    ap.add_argument("--batch", type=int, default=1)
    ap.add_argument("--context", type=int, default=1024, help="tokens in the cache before the timed steps")
    ap.add_argument("--kv", choices=sorted(nf4.KV_FORMATS), default="nf4")
    ap.add_argument("--steps", type=int, default=50)
    a = ap.parse_args()
    cfg = Config(layers=a.layers, batch=a.batch, kv=a.kv, max_len=a.context + a.steps + 16)
    model = Decoder(cfg)
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn((cfg.batch, cfg.hidden), generator=g, device="cuda").to(torch.bfloat16)
    # the context: random keys and values, written as a prompt's would be
    for layer in model.layers:
        n = cfg.batch * a.context
        pos = torch.arange(a.context, device="cuda")
        slots = (model.page_table[:, pos // cfg.page_size].long() * cfg.page_size + pos % cfg.page_size).reshape(-1)
        kv = [torch.randn((n, cfg.kv_heads, cfg.head_dim), generator=g, device="cuda").to(torch.bfloat16) for _ in "kv"]
        nf4.nf4_kv_append(layer.cache, *kv, slots)
    model.lengths.fill_(a.context)
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        model.step(x)  # first calls outside the capture
    side.synchronize()
    model.lengths.fill_(a.context)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        model.step(x)
    for _ in range(3):
        graph.replay()
    begin, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    begin.record()
    for _ in range(a.steps):
        graph.replay()
    end.record()
    end.synchronize()
    ms = begin.elapsed_time(end) / a.steps
    assert nf4.nf4_check_device_error() == 0
    print(f"{cfg.layers} layers, batch {cfg.batch}, context {a.context}, cache {cfg.kv}: {ms:.3f} ms a step, "
          f"{cfg.batch / ms * 1e3:.0f} tokens/s")


if __name__ == "__main__":
    main()
