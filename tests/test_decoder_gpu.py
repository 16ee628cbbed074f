"""The example decoder, steps of a small stack, against the same computation in plain 64-bit torch (GPU).

The plain form takes the library's dequantized weights and the cache's values as they are stored (each is
tested on its own); it rounds activations to bf16 where the library's calls do.  A rounding that falls the
other way moves a value by 2^-8, and the layers pass it on: the bound on the norm of the difference is
2^-8 * sqrt(roundings in a row) = 2^-8 * sqrt(9 a layer), with a factor of 2.
"""
import math
import os
import sys

import pytest
import torch

import nf4_weight_only_gb300 as nf4

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))

pytestmark = pytest.mark.gpu


def bf(x):
    return x.to(torch.bfloat16).double()


def values(cache, which, slots):
    out = nf4.kv_read(cache, slots)[0 if which == "k" else 1]
    return out.double()


def plain_step(model, x, length):
    """The step after which every sequence has `length` keys; the cache already holds the new ones."""
    cfg = model.cfg
    pos = torch.full((cfg.batch,), length - 1, dtype=torch.float64, device="cuda")
    angle = pos[:, None] * model.inv_freq.double()
    cos, sin = angle.cos()[:, None], angle.sin()[:, None]

    def rope(t):
        a, b = t.chunk(2, -1)
        return bf(torch.cat((a * cos - b * sin, b * cos + a * sin), -1))

    def lin(t, w):
        return bf(t @ nf4.dequant(*w).double().T)

    def norm(h, w):
        return bf(h / torch.sqrt((h * h).mean(-1, keepdim=True) + cfg.eps) * w.double())

    r, delta = bf(x.double()), None
    for layer in model.layers:
        s = r if delta is None else r + delta
        h, r = norm(s, layer.norm_in), bf(s)
        q = rope(lin(h, layer.q).view(cfg.batch, cfg.q_heads, cfg.head_dim))
        out = []
        for b in range(cfg.batch):
            j = torch.arange(length, device="cuda")
            slots = model.page_table[b, j // cfg.page_size].long() * cfg.page_size + j % cfg.page_size
            k, v = values(layer.cache, "k", slots), values(layer.cache, "v", slots)  # [length, kv heads, dim]
            qb = q[b].view(cfg.kv_heads, -1, cfg.head_dim)
            p = torch.softmax(torch.einsum("hgd,nhd->hgn", qb, k) * cfg.head_dim ** -0.5, -1)
            out.append(torch.einsum("hgn,nhd->hgd", p, v).reshape(-1))
        delta = lin(bf(torch.stack(out)), layer.o)
        s = r + delta
        h, r = norm(s, layer.norm_mid), bf(s)
        gate, up = lin(h, layer.gate), lin(h, layer.up)
        delta = lin(bf(bf(torch.nn.functional.silu(gate)) * up), layer.down)
    return norm(r + delta, model.norm_out)


@pytest.mark.parametrize("kv,batch", [("bf16", 3), ("fp8", 1), ("nf4", 5)])
def test_decoder_steps(kv, batch):
    from decoder import Config, Decoder
    cfg = Config(hidden=512, q_heads=8, kv_heads=2, head_dim=64, inter=1024, layers=3, batch=batch, max_len=80,
                 page_size=16, kv=kv)
    model = Decoder(cfg, seed=5)
    g = torch.Generator(device="cuda").manual_seed(6)
    bound = 2.0 ** -8 * math.sqrt(9 * cfg.layers) * 2
    for n in range(1, 41):
        x = torch.randn((batch, cfg.hidden), generator=g, device="cuda").to(torch.bfloat16)
        got = model.step(x).double()
        if n in (1, 2, 16, 17, 40):
            want = plain_step(model, x, n)
            assert float((got - want).norm() / want.norm()) <= bound
    assert int(model.lengths[0]) == 40 and nf4.nf4_check_device_error() == 0
