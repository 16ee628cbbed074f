"""What the example decoder writes into its caches (GPU): every layer's new keys and values against the k and v projections
of the layer's own input, with the sequences' adapters and the keys' rotation, in plain 64-bit torch.

The bound on the distance, as a share of the vector's norm: that of the decoder's activations (2^-8 * sqrt(roundings in a
row), factor 2, 13 roundings a layer), and what the cache's format rounds.  Of a value v whose vector (of 64, for NF4) has the
largest size m: bf16 nothing more; fp8 half a step of e4m3, 2^-4 |v| or m / 448 * 2^-10, and its product's rounding 2^-8
|v|; NF4 half the widest gap of its table, 0.152 m, its scale's 2^-11 m and 2^-8 |v|.  The same comparison with the usual
mistakes (no adapter, the next adapter, no rotation, keys and values exchanged) has to fail."""
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


def rounding(want, kv):
    """The most that the cache's format changes each value of [batch, heads, head_dim]."""
    if kv == "bf16":
        return torch.zeros_like(want)
    if kv == "fp8":
        most = want.abs().amax(-1, keepdim=True)
        return want.abs() * (2.0 ** -4 + 2.0 ** -8) + most / 448 * 2.0 ** -10
    most = want.unflatten(-1, (-1, 64)).abs().amax(-1, keepdim=True).expand(*want.shape[:-1], -1, 64).flatten(-2)
    return most * (0.152 + 2.0 ** -11) + want.abs() * 2.0 ** -8


class Walk:
    """One step of the decoder in 64 bits over its stored caches, and what each layer should have written."""

    def __init__(self, model, ids, length):
        self.model, self.cfg, self.length = model, model.cfg, length
        angle = torch.full((self.cfg.batch, 1), float(length - 1), dtype=torch.float64, device="cuda") * \
            model.inv_freq.double()
        self.cos, self.sin = angle.cos()[:, None], angle.sin()[:, None]
        self.x = nf4.embed(ids, *model.table)

    def rope(self, t):
        a, b = t.chunk(2, -1)
        return bf(torch.cat((a * self.cos - b * self.sin, b * self.cos + a * self.sin), -1))

    def heads(self, t):
        return t.view(self.cfg.batch, -1, self.cfg.head_dim)

    def lin(self, t, w, lora=None, i=0, shift=0, adapted=True):
        y = bf(t @ nf4.dequant(*w).double().T)
        if self.cfg.adapters and adapted:
            a, b = lora[0][i].double(), lora[1][i].double()
            for row, adapter in enumerate(self.model.adapter_of.tolist()):
                if adapter >= 0:
                    mine = (adapter + shift) % self.cfg.adapters
                    y[row] += float(self.model.lora_scales[adapter]) * (b[mine] @ (a[mine] @ t[row]))
        return bf(y)

    def norm(self, h, w):
        return bf(h / torch.sqrt((h * h).mean(-1, keepdim=True) + self.cfg.eps) * w.double())

    def layers(self):
        """(layer, what its k and v projections see) one after the other."""
        cfg, r, delta = self.cfg, bf(self.x.double()), None
        for layer in self.model.layers:
            qkv, o, gu, down = (getattr(layer, n, None) for n in ("lora_qkv", "lora_o", "lora_gate_up", "lora_down"))
            s = r if delta is None else r + delta
            h, r = self.norm(s, layer.norm_in), bf(s)
            yield layer, h
            q, out = self.rope(self.heads(self.lin(h, layer.q, qkv, 0))), []
            for b in range(cfg.batch):
                j = torch.arange(self.length, device="cuda")
                k, v = (t.double() for t in nf4.kv_read(layer.cache, self.slots(b, j)))
                p = torch.softmax(torch.einsum("hgd,nhd->hgn", q[b].view(cfg.kv_heads, -1, cfg.head_dim), k) *
                                  cfg.head_dim ** -0.5, -1)
                out.append(torch.einsum("hgn,nhd->hgd", p, v).reshape(-1))
            delta = self.lin(bf(torch.stack(out)), layer.o, o)
            s = r + delta
            h, r = self.norm(s, layer.norm_mid), bf(s)
            gate, up = self.lin(h, layer.gate, gu, 0), self.lin(h, layer.up, gu, 1)
            delta = self.lin(bf(bf(torch.nn.functional.silu(gate)) * up), layer.down, down)

    def slots(self, b, j):
        return self.model.page_table[b, j // self.cfg.page_size].long() * self.cfg.page_size + j % self.cfg.page_size


@pytest.mark.parametrize("kv,batch,adapters,rank", [("bf16", 4, 3, 8), ("nf4", 4, 3, 16), ("fp8", 4, 3, 24), ("nf4", 2, 0, 8)])
def test_new_keys_and_values(kv, batch, adapters, rank):
    from decoder import Config, Decoder
    cfg = Config(hidden=512, q_heads=8, kv_heads=2, head_dim=64, inter=1024, layers=3, max_len=40, page_size=16, vocab=1000,
                 kv=kv, batch=batch, adapters=adapters, rank=rank)
    model = Decoder(cfg, seed=5)
    if adapters:
        model.lora_scales.copy_(torch.tensor([1.5, 2.0, 2.5]))
    g = torch.Generator(device="cuda").manual_seed(6)
    model.ids.copy_(torch.arange(batch, dtype=torch.int32) * 11)
    for n in range(1, 35):
        ids = model.ids.clone()
        model.random.copy_(torch.rand(batch, generator=g, device="cuda"))
        model.generate()
        if n not in (1, 2, 16, 17, 34):
            continue
        walk = Walk(model, ids, n)
        for i, (layer, h) in enumerate(walk.layers()):
            slots = torch.cat([walk.slots(b, torch.tensor([n - 1], device="cuda")) for b in range(batch)])
            got = [t.double() for t in nf4.kv_read(layer.cache, slots)]
            qkv = getattr(layer, "lora_qkv", None)

            def projected(**how):
                return [walk.heads(walk.lin(h, w, qkv, j, **how)) for j, w in ((1, layer.k), (2, layer.v))]

            k, v = projected()

            def near(t, want):
                """For every sequence."""
                drift = 2.0 ** -8 * math.sqrt(13 * (i + 1)) * 2
                bound = (drift * want.flatten(1).norm(dim=1) + rounding(want, kv).flatten(1).norm(dim=1)) * 1.1
                return ((t - want).flatten(1).norm(dim=1) <= bound).tolist()

            assert near(got[0], walk.rope(k)) == [True] * batch and near(got[1], v) == [True] * batch, (n, i)
            assert not any(near(got[0], v)) and not any(near(got[1], walk.rope(k)))
            # A pair turned by an angle a moves by 2 sin(a / 2) of itself, so a vector of 32 pairs with the angles
            # p * 10^(-6 i / 32) by 0.23 of its norm at position 1, which NF4's rounding may hide, and by 0.67 at 16.
            if n > 16:
                assert not any(near(got[0], k)) and not any(near(got[1], walk.rope(v)))
            has = [a >= 0 for a in model.adapter_of.tolist()] if adapters else []
            for how in (dict(adapted=False), dict(shift=1)) if adapters else ():
                wrong_k, wrong_v = projected(**how)
                assert near(got[0], walk.rope(wrong_k)) == [not a for a in has]
                assert near(got[1], wrong_v) == [not a for a in has]
    assert nf4.nf4_check_device_error() == 0
