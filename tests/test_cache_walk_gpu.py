"""Cache writes and reads of more items than one step of the grid takes (GPU): exact, against the formats on the CPU.

A step is at most 8 CTAs an SM of 256 / (head_dim / 8) items (a token and kv head each), rounded up so that the heads
divide it; the sizes take two or three steps with a remainder.
"""
import numpy as np
import pytest
import torch

import nf4_weight_only_gb300 as nf4
import oracle
from gpu_util import DEV, Guarded
from test_layer_ops_gpu import FORMATS, TABLE, gen, randn

pytestmark = pytest.mark.gpu
SMS = torch.cuda.get_device_properties(0).multi_processor_count if torch.cuda.is_available() else 152


def stored(fmt, x):
    """Codes (bytes) and scales of bf16 vectors [n, heads, dim], and their values as bf16, worked out on the CPU."""
    n, heads, dim = x.shape
    f = x.float().cpu().numpy()
    if fmt == "bf16":
        return x.cpu().view(torch.uint8), None, x.cpu()
    if fmt == "fp8":
        s = (np.abs(f).max(-1) / np.float32(448)).astype(np.float32)
        with np.errstate(divide="ignore", invalid="ignore"):
            r = np.where(s[..., None] > 0, f / s[..., None], np.float32(0)).astype(np.float32)
        code = torch.from_numpy(np.clip(r, -448, 448)).to(torch.float8_e4m3fn)
        s = torch.from_numpy(s)
        return code.view(torch.uint8), s, (code.float() * s[..., None]).to(torch.bfloat16)
    codes, scales = oracle.default().quantize(f.reshape(-1, dim))
    codes = torch.from_numpy(codes.copy()).view(n, heads, dim // 2)
    scales = torch.from_numpy(scales.view(np.int16).copy()).view(torch.float16).view(n, heads, dim // 64)
    t = torch.tensor(TABLE, dtype=torch.float32)
    v = torch.stack((t[(codes & 15).long()], t[(codes >> 4).long()]), -1).flatten(-2)
    return codes, scales, (v * scales.float().repeat_interleave(64, -1)).to(torch.bfloat16)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("heads,dim,steps", [(3, 64, 2.3), (5, 128, 2.6), (7, 256, 3.4), (12, 128, 2.2), (1, 256, 3.01),
                                             (8, 64, 1.02), (96, 128, 2.5), (1000, 64, 1.9)])
def test_many_steps(fmt, heads, dim, steps):
    tokens = int(steps * 8 * SMS * (256 // (dim // 8)) / heads) + 1
    page = 48
    pages = tokens // page + 3
    c = nf4.KVCache.empty(fmt, pages, heads, page, dim, DEV)
    arrays = [t for t in (c.k, c.v, c.k_scales, c.v_scales) if t is not None]
    for i, t in enumerate(arrays):
        t.view(torch.uint8).fill_(17 * i + 5)
    before = [t.clone() for t in arrays]
    k, v = randn((tokens, heads, dim), 1), randn((tokens, heads, dim), 2, 3.0)
    k[::97] = 0
    slots = torch.randperm(pages * page, generator=gen(3), device=DEV)[:tokens]
    given = slots.clone()
    given[::11] = -1 - given[::11]
    nf4.nf4_kv_append(c, k, v, given)
    assert nf4.nf4_check_device_error() == 0
    live = (given >= 0).cpu()
    at = slots.cpu()[live]
    p, o = at // page, at % page
    values = []
    for i, x in enumerate((k, v)):
        codes, scales, value = stored(fmt, x)
        values.append(value)
        want = before[i].cpu()
        want.view(torch.uint8)[p, :, o] = codes[live]
        assert torch.equal(arrays[i].cpu().view(torch.uint8), want.view(torch.uint8))
        if scales is not None:
            want = before[i + 2].cpu()
            want[p, :, o] = scales[live]
            assert torch.equal(arrays[i + 2].cpu().view(torch.uint8), want.view(torch.uint8))
    # back, in another order, with skipped ones
    order = torch.randperm(tokens, generator=gen(4), device=DEV)
    ko, vo = Guarded(k.shape, torch.bfloat16), Guarded(v.shape, torch.bfloat16)
    nf4.nf4_kv_read(c, given[order], ko.t, vo.t)
    assert ko.canaries_intact() and vo.canaries_intact() and nf4.nf4_check_device_error() == 0
    for out, value in ((ko.t, values[0]), (vo.t, values[1])):
        value[~live] = 0
        assert torch.equal(out.cpu(), value[order.cpu()])
