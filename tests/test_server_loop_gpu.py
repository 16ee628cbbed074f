"""The example decoder as a server runs it (GPU): plan, embed, layers with adapters, head, sample, and the sampled tokens
are the next step's ids.  Every step's indices are checked against a count on the host, its activations against
plain 64-bit torch with the library's dequantized weights and stored cache values, its tokens against their
definition on the step's own logits.  The bound on the activations is that of the decoder without adapters (2^-8 *
sqrt(roundings in a row), factor 2): an adapter adds one rounding to each linear's, so 13 a layer instead of 9."""
import math
import os
import sys

import pytest
import torch

import nf4_weight_only_gb300 as nf4

from test_sample_gpu import definition

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))

pytestmark = pytest.mark.gpu


def bf(x):
    return x.to(torch.bfloat16).double()


def plain_step(model, x, length):
    cfg = model.cfg
    angle = torch.full((cfg.batch, 1), float(length - 1), dtype=torch.float64, device="cuda") * model.inv_freq.double()
    cos, sin = angle.cos()[:, None], angle.sin()[:, None]

    def rope(t):
        a, b = t.chunk(2, -1)
        return bf(torch.cat((a * cos - b * sin, b * cos + a * sin), -1))

    def lin(t, w, lora, i):
        y = bf(t @ nf4.dequant(*w).double().T)
        if cfg.adapters:
            a, b = lora[0][i].double(), lora[1][i].double()
            for row, adapter in enumerate(model.adapter_of.tolist()):
                if adapter >= 0:
                    y[row] += float(model.lora_scales[adapter]) * (b[adapter] @ (a[adapter] @ t[row]))
        return bf(y)

    def norm(h, w):
        return bf(h / torch.sqrt((h * h).mean(-1, keepdim=True) + cfg.eps) * w.double())

    r, delta = bf(x.double()), None
    for layer in model.layers:
        qkv, o, gu, down = (getattr(layer, n, None) for n in ("lora_qkv", "lora_o", "lora_gate_up", "lora_down"))
        s = r if delta is None else r + delta
        h, r = norm(s, layer.norm_in), bf(s)
        q = rope(lin(h, layer.q, qkv, 0).view(cfg.batch, cfg.q_heads, cfg.head_dim))
        out = []
        for b in range(cfg.batch):
            j = torch.arange(length, device="cuda")
            slots = model.page_table[b, j // cfg.page_size].long() * cfg.page_size + j % cfg.page_size
            k, v = (t.double() for t in nf4.kv_read(layer.cache, slots))
            p = torch.softmax(torch.einsum("hgd,nhd->hgn", q[b].view(cfg.kv_heads, -1, cfg.head_dim), k) *
                              cfg.head_dim ** -0.5, -1)
            out.append(torch.einsum("hgn,nhd->hgd", p, v).reshape(-1))
        delta = lin(bf(torch.stack(out)), layer.o, o, 0)
        s = r + delta
        h, r = norm(s, layer.norm_mid), bf(s)
        gate, up = lin(h, layer.gate, gu, 0), lin(h, layer.up, gu, 1)
        delta = lin(bf(bf(torch.nn.functional.silu(gate)) * up), layer.down, down, 0)
    return norm(r + delta, model.norm_out)


def config(**more):
    from decoder import Config
    return Config(hidden=512, q_heads=8, kv_heads=2, head_dim=64, inter=1024, layers=2, max_len=40, page_size=16,
                  vocab=1000, **more)


@pytest.mark.parametrize("kv,batch,adapters,rank", [("bf16", 3, 2, 8), ("nf4", 5, 3, 16), ("fp8", 1, 0, 8)])
def test_generated_steps(kv, batch, adapters, rank):
    from decoder import Decoder
    model = Decoder(config(kv=kv, batch=batch, adapters=adapters, rank=rank), seed=3)
    cfg = model.cfg
    g = torch.Generator(device="cuda").manual_seed(4)
    bound = 2.0 ** -8 * math.sqrt(13 * cfg.layers) * 2
    model.ids.copy_(torch.arange(batch, dtype=torch.int32) * 7)
    for n in range(1, 36):
        ids = model.ids.clone()
        model.random.copy_(torch.rand(batch, generator=g, device="cuda"))
        model.generate()
        assert model.positions.tolist() == [n - 1] * batch and model.lengths.tolist() == [n] * batch
        assert model.sequences.tolist() == list(range(batch))
        at = [int(model.page_table[b, (n - 1) // 16]) * 16 + (n - 1) % 16 for b in range(batch)]
        assert model.slots.tolist() == at and len(set(at)) == batch
        if n in (1, 2, 16, 17, 35):
            want = plain_step(model, nf4.embed(ids, *model.table), n)
            assert float((model.out.double() - want).norm() / want.norm()) <= bound
        logits = model.logits.float().cpu().numpy()
        for b in range(batch):
            token, _, near = definition(logits[b], float(model.random[b]), float(model.temperature[b]),
                                        int(model.top_k[b]), float(model.top_p[b]))
            assert near < 1e-9 or int(model.ids[b]) == token
    assert nf4.nf4_check_device_error() == 0


def test_captured_generation_is_the_eager_one():
    from decoder import Decoder
    cfg = config(kv="nf4", batch=4, adapters=2, rank=16)
    randoms = torch.rand((30, 4), generator=torch.Generator(device="cuda").manual_seed(9), device="cuda")
    runs = []
    for captured in (False, True):
        model, ids = Decoder(cfg, seed=2), []
        step = model.generate
        if captured:
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                model.generate()
            step = graph.replay
        for u in randoms:
            model.random.copy_(u)
            step()
            ids.append(model.ids.tolist())
        runs.append((ids, model.lengths.tolist(), model.page_table.tolist(), model.free_state.tolist()))
    assert runs[0] == runs[1]
    assert len({tuple(x) for x in runs[0][0]}) > 5 and nf4.nf4_check_device_error() == 0
