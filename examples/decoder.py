"""A decoder at decode time, built from the library's calls: the step's indices, NF4 linears with low-rank
adapters of the requests beside them, residual norms, rotary positions, a paged (quantised) key-value cache, the
attention of one new token over it, and the choice of the next token.

    python examples/decoder.py --layers 36 --batch 1 --context 1024 --kv nf4
    python examples/decoder.py --batch 32 --adapters 8 --rank 16 --vocab 151936

builds a 3B-shaped stack with random weights, fills the cache to the given context and reports the time of a
decode step replayed as one CUDA graph.  The step is what a serving loop would run: pages are taken from the
pool as sequences grow, and with a vocabulary the sampled tokens are the next replay's ids.
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

        def adapters(*linears):
            """(A, B) of every loaded adapter for linears that share their input."""
            sides = [], []
            for codes, _ in linears:
                n, k = codes.shape[0], 2 * codes.shape[1]
                for side, shape, scale in zip(sides, ((cfg.rank, k), (n, cfg.rank)), (k ** -0.5, cfg.rank ** -0.5)):
                    w = torch.randn((cfg.adapters, *shape), generator=generator, device="cuda") * scale
                    side.append(w.to(torch.bfloat16))
            return sides

        if cfg.adapters:
            self.lora_qkv, self.lora_o = adapters(self.q, self.k, self.v), adapters(self.o)
            self.lora_gate_up, self.lora_down = adapters(self.gate, self.up), adapters(self.down)
        self.cache = nf4.KVCache.empty(cfg.kv, cfg.pages(), cfg.kv_heads, cfg.page_size, cfg.head_dim)


class Config:
    def __init__(self, hidden=2048, q_heads=16, kv_heads=2, head_dim=128, inter=11008, layers=36, batch=1, max_len=2048,
                 page_size=64, kv="nf4", theta=1e6, eps=1e-6, adapters=0, rank=16, vocab=0):
        self.__dict__.update(locals())

    def pages(self):
        return self.batch * -(-self.max_len // self.page_size)


class Decoder:
    def __init__(self, cfg: Config, seed: int = 0):
        self.cfg = cfg
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.layers = [Layer(cfg, g) for _ in range(cfg.layers)]
        self.norm_out = torch.ones(cfg.hidden, dtype=torch.bfloat16, device="cuda")
        half = cfg.head_dim // 2
        self.inv_freq = (cfg.theta ** (-torch.arange(half, dtype=torch.float64, device="cuda") / half)).float()

        def ints(*shape, dtype=torch.int32):
            return torch.zeros(shape, dtype=dtype, device="cuda")

        # the pool of pages, and what a step's plan writes: every sequence brings one token
        self.free_pages, self.free_state = nf4.free_ring(cfg.pages())
        self.page_table, self.lengths = ints(cfg.batch, -(-cfg.max_len // cfg.page_size)), ints(cfg.batch)
        self.new_tokens = torch.ones(cfg.batch, dtype=torch.int32, device="cuda")
        self.starts, self.slots = ints(cfg.batch + 1), ints(cfg.batch, dtype=torch.int64)
        self.positions, self.sequences = ints(cfg.batch), ints(cfg.batch)
        if cfg.adapters:  # the adapter of each sequence (-1: none)
            self.adapter_of = torch.arange(cfg.batch, dtype=torch.int32, device="cuda") % (cfg.adapters + 1) - 1
            self.lora_scales = torch.full((cfg.adapters,), 0.5, device="cuda")
            self.lora_plan = nf4.lora_plan_buffer(cfg.batch, cfg.adapters)
            self.lora_workspace = nf4.lora_workspace(cfg.batch, cfg.adapters, cfg.rank, 3)
        if cfg.vocab:  # one packed table for the embedding and the head
            w = torch.randn((cfg.vocab, cfg.hidden), generator=g, device="cuda") * cfg.hidden ** -0.5
            self.table = nf4.quantize(w)
            self.ids, self.random = ints(cfg.batch), torch.zeros(cfg.batch, device="cuda")
            self.temperature = torch.full((cfg.batch,), 0.8, device="cuda")
            self.top_k, self.top_p = ints(cfg.batch) + 50, torch.full((cfg.batch,), 0.95, device="cuda")
            self.x = torch.empty((cfg.batch, cfg.hidden), dtype=torch.bfloat16, device="cuda")
            self.logits = torch.empty((cfg.batch, cfg.vocab), dtype=torch.bfloat16, device="cuda")
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
        nf4.nf4_plan_step(self.lengths, self.new_tokens, cfg.page_size, self.page_table, self.free_pages, self.free_state,
                          self.free_state, self.lengths, self.starts, self.slots, self.positions, self.sequences)
        slots, positions = self.slots, self.positions[None]  # the same in every layer
        if cfg.adapters:
            nf4.nf4_lora_plan(self.adapter_of, cfg.adapters, self.lora_plan, sequences=self.sequences)
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
            self.adapt(layer, "lora_qkv", self.h, self.q.view(flat), self.k.view(flat), self.v.view(flat))
            nf4.nf4_rope(self.q, self.k, positions, self.inv_freq, self.q, self.k)
            nf4.nf4_kv_append(layer.cache, self.k, self.v, slots)
            nf4.nf4_attention_decode(layer.cache, self.q, self.page_table, self.lengths, self.attn, self.workspace)
            nf4.nf4_linear(self.attn.view(flat), *layer.o, self.delta)
            self.adapt(layer, "lora_o", self.attn.view(flat), self.delta)
            nf4.nf4_rmsnorm(self.delta, layer.norm_mid, cfg.eps, residual=self.residual, residual_out=self.residual,
                            y=self.h)
            nf4.nf4_linear_grouped(self.h, [layer.gate[0], layer.up[0]], [layer.gate[1], layer.up[1]],
                                   [self.gate, self.up])
            self.adapt(layer, "lora_gate_up", self.h, self.gate, self.up)
            inner = torch.nn.functional.silu(self.gate) * self.up
            nf4.nf4_linear(inner, *layer.down, self.delta)
            self.adapt(layer, "lora_down", inner, self.delta)
        nf4.nf4_rmsnorm(self.delta, self.norm_out, cfg.eps, residual=self.residual, residual_out=self.residual,
                        y=self.out)
        return self.out

    def adapt(self, layer: Layer, name: str, x: torch.Tensor, *ys: torch.Tensor) -> None:
        """Adds the sequences' adapters to what linears made of x."""
        if self.cfg.adapters:
            a, b = getattr(layer, name)
            nf4.nf4_lora(x, self.lora_plan, self.lora_scales, a, b, list(ys), self.lora_workspace)

    def generate(self) -> torch.Tensor:
        """One token of every sequence from its last one: ids -> ids, drawn with self.random."""
        nf4.nf4_embed(self.ids, *self.table, self.x)
        nf4.nf4_linear(self.step(self.x), *self.table, self.logits)
        nf4.nf4_sample(self.logits, self.random, self.ids, self.temperature, self.top_k, self.top_p)
        return self.ids


def main():
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--layers", type=int, default=36)
    ap.add_argument("--batch", type=int, default=1)
    ap.add_argument("--context", type=int, default=1024, help="tokens in the cache before the timed steps")
    ap.add_argument("--kv", choices=sorted(nf4.KV_FORMATS), default="nf4")
    ap.add_argument("--steps", type=int, default=50)
    ap.add_argument("--adapters", type=int, default=0, help="low-rank adapters that the sequences take turns at")
    ap.add_argument("--rank", type=int, default=16)
    ap.add_argument("--vocab", type=int, default=0, help="sample tokens and feed them back (0: steps alone)")
    a = ap.parse_args()
    cfg = Config(layers=a.layers, batch=a.batch, kv=a.kv, max_len=a.context + a.steps + 16, adapters=a.adapters,
                 rank=a.rank, vocab=a.vocab)
    model = Decoder(cfg)
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn((cfg.batch, cfg.hidden), generator=g, device="cuda").to(torch.bfloat16)
    # the context: random keys and values, written as a prompt's would be
    n = cfg.batch * a.context
    slots = torch.empty(n, dtype=torch.int64, device="cuda")
    rows = [torch.empty(n, dtype=torch.int32, device="cuda") for _ in ("positions", "sequences")]
    nf4.nf4_plan_step(model.lengths, model.new_tokens * a.context, cfg.page_size, model.page_table, model.free_pages,
                      model.free_state, model.free_state, model.lengths, model.starts, slots, *rows)
    for layer in model.layers:
        kv = [torch.randn((n, cfg.kv_heads, cfg.head_dim), generator=g, device="cuda").to(torch.bfloat16) for _ in "kv"]
        nf4.nf4_kv_append(layer.cache, *kv, slots)

    def once():
        if cfg.vocab:
            model.random.uniform_()
            model.generate()
        else:
            model.step(x)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        once()  # first calls outside the capture
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        once()
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
    more = (f", {cfg.adapters} adapters of rank {cfg.rank}" if cfg.adapters else "") + (
        f", {cfg.vocab} tokens to choose from" if cfg.vocab else "")
    print(f"{cfg.layers} layers, batch {cfg.batch}, context {a.context}, cache {cfg.kv}{more}: {ms:.3f} ms a step, "
          f"{cfg.batch / ms * 1e3:.0f} tokens/s")


if __name__ == "__main__":
    main()
