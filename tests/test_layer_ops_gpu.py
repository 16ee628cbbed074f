"""Cache, attention, rotary and norm kernels against plain 64-bit implementations (GPU).

Tolerances, from the arithmetic:
  attention   the weights may be rounded to bf16 before the product with V (2^-9 relative each) and the
              V codes to fp16 (2^-12); a score may be off by A 2^-12 from rounding K's code values to
              fp16, A = max_j scale * sum_d |q_d k_jd|, which moves a softmax weight by twice that.  So
              |o - o64| <= 2^-8 |o64| + (2^-8 + 2^-11 A) * sum_j p_j |v_j|, the first term for bf16.
  rope        2^-8 |o| for bf16, and 2^-18 (|x| + |y|) for the sine and cosine (2^-20 absolute each)
  norm        2^-8 |y| for bf16; the row scale 2^-20 relative; an 8-bit value is within half an e4m3
              step of y: 2^-4 |y| (normal) or 2^-10 s (below 2^-6 s), and 2^-10 more for its inputs
Quantized codes and scales of the cache, and values read back, are exact.
"""
import numpy as np
import pytest
import torch

import nf4_weight_only_gb300 as nf4
import oracle
from gpu_util import DEV, Guarded, dev_to_bits

pytestmark = pytest.mark.gpu
FORMATS = ("bf16", "fp8", "nf4")
TABLE = [-1.0, -0.6961928009986877, -0.5250730514526367, -0.39491748809814453, -0.28444138169288635,
         -0.18477343022823334, -0.09105003625154495, 0.0, 0.07958029955625534, 0.16093020141124725,
         0.24611230194568634, 0.33791524171829224, 0.44070982933044434, 0.5626170039176941,
         0.7229568362236023, 1.0]


def gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def randn(shape, seed, scale=1.0):
    return (torch.randn(shape, generator=gen(seed), device=DEV) * scale).to(torch.bfloat16)


def new_cache(fmt, pages, heads, page, dim, seed=None):
    """A cache; with a seed, every place holds data."""
    c = nf4.KVCache.empty(fmt, pages, heads, page, dim, DEV)
    if seed is not None:
        n = pages * page
        nf4.nf4_kv_append(c, randn((n, heads, dim), seed), randn((n, heads, dim), seed + 1),
                          torch.arange(n, device=DEV))
    return c


def values64(c, which):
    """The cache's values in 64 bits, [pages, heads, page, dim]."""
    x, s = (c.k, c.k_scales) if which == "k" else (c.v, c.v_scales)
    if c.format == "bf16":
        return x.double()
    if c.format == "fp8":
        return x.float().double() * s.double()[..., None]
    t = torch.tensor(TABLE, dtype=torch.float64, device=DEV)
    v = torch.stack((t[(x & 15).long()], t[(x >> 4).long()]), -1).flatten(-2)
    return v * s.double().repeat_interleave(64, -1)


def poison(c, keep):
    """NaN in every place outside the bool mask keep [pages, page] (codes, values and scales)."""
    gone = ~keep
    for x, s in ((c.k, c.k_scales), (c.v, c.v_scales)):
        raw = x.view(torch.uint8)
        raw.permute(0, 2, 1, 3)[gone] = 0xFF if c.format != "fp8" else 0x7F  # bf16 0xFFFF and e4m3 0x7F are NaN
        if s is not None:
            s.transpose(1, 2)[gone] = float("nan")


# ---------------------------------------------------------------------------------------------
# Writing and reading the cache
# ---------------------------------------------------------------------------------------------
def awkward(tokens, heads, dim, seed):
    """Vectors with the cases a quantiser can go wrong at: zeros, ties, tiny and large values."""
    x = randn((tokens, heads, dim), seed).float()
    flat = x.view(-1, dim)
    n = flat.shape[0]
    if n > 6:
        flat[0] = 0
        flat[1] = -0.0
        flat[2] *= 1e-38
        flat[3] *= 1e-41
        flat[4] *= 1e30
        flat[5, :64] = 0
        flat[6] = torch.linspace(-1, 1, dim, device=DEV)
    return x.to(torch.bfloat16)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("tokens,heads,page,dim", [(1, 1, 16, 64), (7, 3, 48, 128), (65, 8, 16, 128), (130, 2, 256, 256),
                                                   (300, 5, 32, 64), (0, 2, 16, 128)])
def test_append_is_exact_and_touches_only_its_places(fmt, tokens, heads, page, dim):
    pages = tokens // page + 3
    c = new_cache(fmt, pages, heads, page, dim, seed=5)
    before = [t.clone() for t in (c.k, c.v, c.k_scales, c.v_scales) if t is not None]
    k, v = awkward(tokens, heads, dim, 7), awkward(tokens, heads, dim, 8)
    slots = torch.randperm(pages * page, generator=gen(9), device=DEV)[:tokens]
    skipped = slots.clone()
    skipped[::5] = -1
    nf4.nf4_kv_append(c, k, v, skipped)
    assert nf4.nf4_check_device_error() == 0
    slots, k, v = slots[skipped >= 0], k[skipped >= 0], v[skipped >= 0]
    p, o = slots // page, slots % page
    want = [t.clone() for t in before]
    n = 0
    for x in (k, v):
        if fmt == "bf16":
            want[n].view(torch.int16)[p, :, o] = x.view(torch.int16)
        elif fmt == "fp8":
            f = x.float().cpu().numpy()
            s = (np.abs(f).max(-1) / np.float32(448)).astype(np.float32) if f.size else np.zeros(f.shape[:2], np.float32)
            with np.errstate(divide="ignore", invalid="ignore"):
                r = np.where(s[..., None] > 0, f / s[..., None], np.float32(0)).astype(np.float32)
            code = torch.from_numpy(np.clip(r, -448, 448)).to(torch.float8_e4m3fn).view(torch.uint8).to(DEV)
            want[n].view(torch.uint8)[p, :, o] = code
            want[n + 2][p, :, o] = torch.from_numpy(s).to(DEV)
        else:
            f = x.float().cpu().numpy().reshape(-1, dim)
            codes, scales = oracle.default().quantize(f) if f.size else (np.zeros((0, dim // 2), np.uint8),
                                                                       np.zeros((0, dim // 64), np.uint16))
            want[n][p, :, o] = torch.from_numpy(codes.copy()).to(DEV).view(-1, heads, dim // 2)
            sc = torch.from_numpy(scales.view(np.int16).copy()).to(DEV).view(torch.float16).view(-1, heads, dim // 64)
            want[n + 2][p, :, o] = sc
        n += 1
    got = [t for t in (c.k, c.v, c.k_scales, c.v_scales) if t is not None]
    for a, b in zip(got, want):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))


def test_nf4_append_equals_quantize_at_every_threshold():
    """bf16 values dense around each decision threshold, for many group maxima."""
    rows = 2048
    top = (1 + torch.rand(rows, 1, generator=gen(1), device=DEV)).to(torch.bfloat16).float()
    t = torch.tensor(TABLE, device=DEV)
    mid = (t[1:] + t[:-1]) / 2
    x = (mid.repeat(9)[:127] * (1 + torch.randn(rows, 127, generator=gen(2), device=DEV) * 2e-3)) * top
    x = torch.cat((x[:, :63], top, x[:, 63:126], -top), 1).to(torch.bfloat16)
    c = nf4.KVCache.empty("nf4", rows // 16, 1, 16, 128, DEV)
    nf4.nf4_kv_append(c, x.view(rows, 1, 128), x.view(rows, 1, 128), torch.arange(rows, device=DEV))
    codes, scales = nf4.quantize(x.float())
    assert torch.equal(c.k.view(rows, 64), codes) and torch.equal(c.v.view(rows, 64), codes)
    assert torch.equal(c.k_scales.view(rows, 2).view(torch.int16), scales.view(torch.int16))


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("tokens,heads,page,dim", [(1, 1, 16, 64), (33, 3, 48, 128), (500, 2, 32, 256), (0, 2, 16, 64)])
def test_read_back_is_exact(fmt, tokens, heads, page, dim):
    c = new_cache(fmt, 12, heads, page, dim, seed=3)
    slots = torch.randint(0, 12 * page, (tokens,), generator=gen(4), device=DEV)
    slots[1::7] = -3
    ko, vo = Guarded((tokens, heads, dim), torch.bfloat16), Guarded((tokens, heads, dim), torch.bfloat16)
    nf4.nf4_kv_read(c, slots, ko.t, vo.t)
    assert ko.canaries_intact() and vo.canaries_intact() and nf4.nf4_check_device_error() == 0
    at = slots.clamp_min(0)
    for out, which, x, s in ((ko.t, "k", c.k, c.k_scales), (vo.t, "v", c.v, c.v_scales)):
        f = values64(c, which)  # a code value times a scale: the product in 64 bits is exact
        want = f[at // page, :, at % page].float().to(torch.bfloat16)
        want[slots < 0] = 0
        assert torch.equal(out, want)
    only = torch.empty((tokens, heads, dim), dtype=torch.bfloat16, device=DEV)
    nf4.nf4_kv_read(c, slots, None, only)
    assert torch.equal(only, vo.t)


@pytest.mark.parametrize("fmt", FORMATS)
def test_slots_outside_the_cache_are_reported(fmt):
    c = new_cache(fmt, 2, 2, 16, 64, seed=1)
    before = c.k.clone()
    x = randn((3, 2, 64), 2)
    nf4.nf4_kv_append(c, x, x, torch.tensor([32, 1 << 40, -1], device=DEV))
    assert nf4.nf4_check_device_error() == 42 and torch.equal(c.k.view(torch.uint8), before.view(torch.uint8))
    k, v = nf4.kv_read(c, torch.tensor([0, 32, 1 << 62], device=DEV))
    assert nf4.nf4_check_device_error() == 42
    assert not k[1:].any() and not v[1:].any() and k[0].any()
    assert nf4.nf4_check_device_error() == 0


# ---------------------------------------------------------------------------------------------
# Attention
# ---------------------------------------------------------------------------------------------
def paged(lengths, page, pages, max_pages, seed, fill=-7):
    """A page table with the sequences' pages scattered over the cache, `fill` in unused entries."""
    order = torch.randperm(pages, generator=torch.Generator().manual_seed(seed)).tolist()
    table = torch.full((len(lengths), max_pages), fill, dtype=torch.int32)
    for b, n in enumerate(lengths):
        for j in range(-(-max(0, n) // page)):
            table[b, j] = order.pop()
    return table


def reference(c, q, table, lengths, scale, window, skip_bad=False):
    """64-bit attention: outputs, and the tolerance of each."""
    k, v = values64(c, "k"), values64(c, "v")
    bsz, hq, d = q.shape
    group = hq // c.kv_heads
    out = torch.zeros((bsz, hq, d), dtype=torch.float64, device=DEV)
    tol = torch.zeros_like(out)
    for b, n in enumerate(lengths):
        n = min(max(n, 0), table.shape[1] * c.page_size)
        j = torch.arange(max(0, n - window) if window else 0, n, device=DEV)
        if skip_bad:
            page_ok = (table[b] >= 0) & (table[b] < c.pages)
            j = j[page_ok.to(DEV)[j // c.page_size]]
        if not len(j):
            continue
        pages = table[b].to(DEV)[j // c.page_size].long()
        kk, vv = k[pages, :, j % c.page_size].transpose(0, 1), v[pages, :, j % c.page_size].transpose(0, 1)
        qq = q[b].double().view(c.kv_heads, group, d)
        p = torch.softmax(qq @ kk.transpose(1, 2) * scale, -1)
        out[b] = (p @ vv).reshape(hq, d)
        big = (qq.abs() @ kk.abs().transpose(1, 2)).amax(-1, keepdim=True) * abs(scale)
        tol[b] = (2.0 ** -8 * (p @ vv).abs() + (2.0 ** -8 + 2.0 ** -11 * big) * (p @ vv.abs())).reshape(hq, d)
    return out, tol


def check(c, q, table, lengths, scale=None, window=0, ws=None, skip_bad=False, error=0):
    scale = c.head_dim ** -0.5 if scale is None else scale
    ws = nf4.attention_workspace(c, q.shape[0], q.shape[1]) if ws is None else ws
    out = Guarded(q.shape, torch.bfloat16)
    out.t.fill_(float("nan"))
    n = torch.tensor(lengths, dtype=torch.int32, device=DEV)
    nf4.nf4_attention_decode(c, q, table.to(DEV), n, out.t, ws, scale=scale, window=window)
    assert nf4.nf4_check_device_error() == error
    assert out.canaries_intact()
    want, tol = reference(c, q, table, lengths, scale, window, skip_bad)
    off = (out.t.double() - want).abs()
    assert bool((off <= tol).all()), f"off by {float((off / tol.clamp_min(1e-300)).max())} of the tolerance"
    return out.t


LENGTHS = [0, 1, 15, 16, 17, 31, 33, 47, 48, 49, 64, 100, 127, 129, 257, 511, 700]


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("heads,group,page,dim", [(1, 1, 16, 64), (2, 8, 16, 128), (3, 5, 48, 128), (2, 6, 64, 256),
                                                  (1, 12, 32, 64), (2, 16, 16, 128), (1, 20, 128, 128), (1, 33, 16, 256),
                                                  (8, 2, 256, 64), (4, 3, 16, 256)])
def test_attention_ragged(fmt, heads, group, page, dim):
    need = sum(-(-n // page) for n in LENGTHS)
    c = new_cache(fmt, need + 2, heads, page, dim, seed=11)
    table = paged(LENGTHS, page, need + 2, -(-700 // page) + 1, 12)
    keep = torch.zeros((need + 2, page), dtype=torch.bool, device=DEV)
    for b, n in enumerate(LENGTHS):
        j = torch.arange(n)
        keep[table[b][j // page].long().to(DEV), (j % page).to(DEV)] = True
    q = randn((len(LENGTHS), heads * group, dim), 13, 2.0)
    first = check(c, q, table, LENGTHS)
    poison(c, keep)
    out = nf4.attention_decode(c, q, table.to(DEV), torch.tensor(LENGTHS, dtype=torch.int32, device=DEV),
                               nf4.attention_workspace(c, len(LENGTHS), heads * group))
    assert torch.equal(out, first)  # what is not attended to does not matter, bit for bit


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("window", [1, 5, 16, 17, 100, 300, 5000])
def test_attention_window(fmt, window):
    lengths = [0, 1, 5, 16, 40, 101, 316, 317, 318, 1000]
    page = 32
    need = sum(-(-n // page) for n in lengths)
    c = new_cache(fmt, need, 2, page, 128, seed=21)
    table = paged(lengths, page, need, 40, 22)
    q = randn((len(lengths), 10, 128), 23)
    check(c, q, table, lengths, window=window)
    # pages wholly before the window need not be there, and what precedes it may be NaN
    keep = torch.ones((need, page), dtype=torch.bool, device=DEV)
    for b, n in enumerate(lengths):
        j = torch.arange(max(0, n - window))
        keep[table[b][j // page].long().to(DEV), (j % page).to(DEV)] = False
    want, tol = reference(c, q, table, lengths, 128 ** -0.5, window)
    poison(c, keep)
    for b, n in enumerate(lengths):
        table[b, :max(0, n - window) // page] = -1
    n = torch.tensor(lengths, dtype=torch.int32, device=DEV)
    out = nf4.attention_decode(c, q, table.to(DEV), n, nf4.attention_workspace(c, 10, 10), window=window)
    assert nf4.nf4_check_device_error() == 0
    assert bool(((out.double() - want).abs() <= tol).all())


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("batch,heads,group,dim,length", [(1, 2, 8, 128, 40001), (1, 1, 1, 64, 9973), (3, 1, 16, 256, 5003),
                                                          (1, 8, 5, 128, 3001), (40, 4, 4, 128, 613), (300, 2, 2, 64, 37)])
def test_attention_split_and_joined(fmt, batch, heads, group, dim, length):
    page = 64
    lengths = [max(1, length - 3 * b) for b in range(batch)]
    need = sum(-(-n // page) for n in lengths)
    c = new_cache(fmt, need, heads, page, dim, seed=31)
    table = paged(lengths, page, need, -(-length // page), 32)
    q = randn((batch, heads * group, dim), 33)
    ws = nf4.attention_workspace(c, batch, heads * group)
    first = check(c, q, table, lengths, ws=ws)
    for _ in range(5):  # the same bytes each time, from the workspace as the last call left it
        again = nf4.attention_decode(c, q, table.to(DEV), torch.tensor(lengths, dtype=torch.int32, device=DEV), ws)
        assert torch.equal(again, first)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("scale", [0.0, 1.0, 30.0, -2.0])
def test_attention_scales(fmt, scale):
    """Scores from all equal to one key taking everything."""
    c = new_cache(fmt, 20, 2, 16, 128, seed=41)
    lengths = [300, 77]
    table = torch.arange(20, dtype=torch.int32).view(1, 20).repeat(2, 1)
    check(c, randn((2, 8, 128), 42), table, lengths, scale=scale)


@pytest.mark.parametrize("fmt", ("fp8", "nf4"))
@pytest.mark.parametrize("factor", [1e-6, 1e-3, 1e3])
def test_attention_value_range(fmt, factor):
    """V far from one, with single tokens far larger than the rest; K and q far apart in size."""
    n, page = 600, 16
    c = nf4.KVCache.empty(fmt, 40, 1, page, 128, DEV)
    wide = max(factor, 1e-3) if fmt == "nf4" else factor  # an fp16 scale holds no absmax past 65504
    k, v = randn((n, 1, 128), 51, 1 / wide), randn((n, 1, 128), 52, min(factor, 100.0) if fmt == "nf4" else factor)
    v[100] *= 30
    v[599] *= 50
    v[300] = 0
    nf4.nf4_kv_append(c, k, v, torch.arange(n, device=DEV))
    table = torch.arange(40, dtype=torch.int32).view(1, 40)
    check(c, randn((1, 8, 128), 53, wide), table, [n])


def test_attention_bad_pages_and_lengths():
    for fmt in FORMATS:
        c = new_cache(fmt, 10, 2, 16, 128, seed=61)
        q = randn((3, 4, 128), 62)
        table = torch.tensor([[0, 1, 2], [3, 10, 4], [-1, 5, 1 << 30]], dtype=torch.int32)
        check(c, q, table, [48, 40, 48], skip_bad=True, error=43)
        check(c, q, table[:1].repeat(3, 1), [49, 1 << 30, 48], error=43)
        check(c, q, table[:1].repeat(3, 1), [-1, -(1 << 31), 48])
        empty = torch.zeros((3, 0), dtype=torch.int32)
        check(c, q, empty, [0, 0, 0])
        nothing = nf4.KVCache.empty(fmt, 0, 2, 16, 128, DEV)
        out = nf4.attention_decode(nothing, q, table.to(DEV), torch.tensor([0, 5, 0], dtype=torch.int32, device=DEV),
                                   nf4.attention_workspace(nothing, 3, 4))
        assert not out.any() and nf4.nf4_check_device_error() == 43


def test_attention_workspace_serves_calls_of_different_sizes():
    big = new_cache("bf16", 700, 2, 16, 128, seed=71)
    small = new_cache("nf4", 64, 4, 16, 64, seed=72)
    ws = torch.zeros(max(nf4.nf4_attention_workspace_bytes(big, 2, 16), nf4.nf4_attention_workspace_bytes(small, 9, 8)),
                     dtype=torch.uint8, device=DEV)
    tb = torch.arange(700, dtype=torch.int32).view(1, 700).repeat(2, 1)
    ts = torch.arange(64, dtype=torch.int32).view(1, 64).repeat(9, 1)
    qb, qs = randn((2, 16, 128), 73), randn((9, 8, 64), 74)
    for i in range(3):
        check(big, qb, tb, [11200, 7000 + i], ws=ws)
        check(small, qs, ts, [1000, 3, 0, 16, 200, 64, 5, 999, 1024 - i], ws=ws)


@pytest.mark.parametrize("fmt", FORMATS)
def test_attention_past_32_bit_offsets(fmt):
    """Pages whose values lie more than 2^31 elements and 2^32 bytes into the cache."""
    vec = {"bf16": 128, "fp8": 64, "nf4": 32}[fmt]
    page, dim = 256, 64
    pages = (1 << 32) // (vec * page) + 4
    c = nf4.KVCache.empty(fmt, pages, 1, page, dim, DEV)
    n = 3 * page
    slots = (pages - 3) * page + torch.arange(n, device=DEV)
    k, v = randn((n, 1, dim), 81), randn((n, 1, dim), 82)
    nf4.nf4_kv_append(c, k, v, slots)
    small = nf4.KVCache.empty(fmt, 3, 1, page, dim, DEV)
    nf4.nf4_kv_append(small, k, v, torch.arange(n, device=DEV))
    q = randn((1, 4, dim), 83)
    lengths = torch.tensor([n - 5], dtype=torch.int32, device=DEV)
    far = nf4.attention_decode(c, q, torch.tensor([[pages - 3, pages - 2, pages - 1]], dtype=torch.int32, device=DEV),
                               lengths, nf4.attention_workspace(c, 1, 4))
    near = nf4.attention_decode(small, q, torch.tensor([[0, 1, 2]], dtype=torch.int32, device=DEV), lengths,
                                nf4.attention_workspace(small, 1, 4))
    assert torch.equal(far, near) and nf4.nf4_check_device_error() == 0
    for a, b in zip(nf4.kv_read(c, slots), nf4.kv_read(small, torch.arange(n, device=DEV))):
        assert torch.equal(a, b)


def test_streams_and_graph_replay():
    """Append and attention on a side stream and in a replayed graph, lengths growing between replays."""
    c = nf4.KVCache.empty("fp8", 64, 2, 16, 128, DEV)
    table = torch.arange(64, dtype=torch.int32, device=DEV).view(2, 32)
    lengths = torch.zeros(2, dtype=torch.int32, device=DEV)
    k, v, q = randn((2, 2, 128), 91), randn((2, 2, 128), 92), randn((2, 8, 128), 93)
    slots = torch.zeros(2, dtype=torch.int64, device=DEV)
    out = torch.empty_like(q)
    ws = nf4.attention_workspace(c, 2, 8)
    side = torch.cuda.Stream()

    def step():
        nf4.nf4_kv_append(c, k, v, slots)
        nf4.nf4_attention_decode(c, q, table, lengths, out, ws)

    def place(n):
        lengths.fill_(n + 1)
        slots.copy_(table[:, n // 16].long() * 16 + n % 16)

    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        place(0)
        step()
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        step()
    for n in range(40):
        place(n)
        k.copy_(randn((2, 2, 128), 1000 + n))
        v.copy_(randn((2, 2, 128), 2000 + n))
        graph.replay()
    want, tol = reference(c, q, table.cpu(), [40, 40], 128 ** -0.5, 0)
    assert bool(((out.double() - want).abs() <= tol).all()) and nf4.nf4_check_device_error() == 0


# ---------------------------------------------------------------------------------------------
# Rotary positions
# ---------------------------------------------------------------------------------------------
def rope64(x, positions, sections, inv_freq, interleaved, magnitude):
    x = x.double()
    n = 2 * inv_freq.shape[0]
    axis = torch.repeat_interleave(torch.arange(len(sections)), torch.tensor(sections)).to(DEV)
    angle = (positions.double()[axis].T * inv_freq.double())[:, None]
    first, second = ((slice(0, n, 2), slice(1, n, 2)) if interleaved else (slice(0, n // 2), slice(n // 2, n)))
    a, b = x[..., first], x[..., second]
    y, tol = x.clone(), torch.zeros_like(x)
    y[..., first] = magnitude * (a * angle.cos() - b * angle.sin())
    y[..., second] = magnitude * (b * angle.cos() + a * angle.sin())
    t = 2.0 ** -18 * abs(magnitude) * (a.abs() + b.abs())
    tol[..., first], tol[..., second] = t, t
    tol[..., :n] += 2.0 ** -8 * y[..., :n].abs()
    return y, tol


@pytest.mark.parametrize("tokens,hq,hk,dim,rotary,sections,inter", [
    (1, 16, 2, 128, 128, (64,), False), (8, 40, 8, 128, 128, (64,), False), (37, 6, 1, 64, 32, (16,), True),
    (301, 48, 8, 128, 128, (22, 21, 21), False), (129, 3, 3, 256, 256, (50, 0, 70, 8), True), (5, 1, 1, 16, 16, (3, 5), False),
    (700, 0, 4, 80, 48, (24,), False), (3000, 32, 8, 128, 64, (11, 21), True), (0, 4, 4, 64, 64, (32,), False),
    (2, 200, 100, 128, 128, (64,), False)])
def test_rope(tokens, hq, hk, dim, rotary, sections, inter):
    q, k = randn((tokens, hq, dim), 1), randn((tokens, hk, dim), 2)
    pos = torch.randint(0, 131072, (len(sections), tokens), generator=gen(3), device=DEV, dtype=torch.int32)
    if tokens > 4:
        pos[:, 0], pos[:, 1], pos[:, 2], pos[0, 3], pos[0, 4] = 0, 2**31 - 1, -(2**31), -5, 1
    inv = (1e6 ** (-torch.arange(rotary // 2, device=DEV, dtype=torch.float64) / (rotary // 2))).float()
    qo, ko = Guarded(q.shape, torch.bfloat16), Guarded(k.shape, torch.bfloat16)
    nf4.nf4_rope(q, k, pos, inv, qo.t, ko.t, sections=list(sections), interleaved=inter, magnitude=1.25)
    assert qo.canaries_intact() and ko.canaries_intact()
    for x, o in ((q, qo.t), (k, ko.t)):
        want, tol = rope64(x, pos, sections, inv, inter, 1.25)
        assert bool(((o.double() - want).abs() <= tol).all())
        assert torch.equal(o[..., rotary:], x[..., rotary:])
    qi, ki = q.clone(), k.clone()
    nf4.nf4_rope(qi, ki, pos, inv, qi, ki, sections=list(sections), interleaved=inter, magnitude=1.25)
    assert torch.equal(qi, qo.t) and torch.equal(ki, ko.t)  # in place
    if hk:
        one = torch.empty_like(k)
        nf4.nf4_rope(None, k, pos, inv, None, one, sections=list(sections), interleaved=inter, magnitude=1.25)
        assert torch.equal(one, ko.t)


def test_rope_keeps_relative_positions():
    """q . k after rotation depends on the distance of the positions only (to the outputs' rounding)."""
    q, k = randn((1, 1, 128), 1), randn((1, 1, 128), 2)
    inv = (1e4 ** (-torch.arange(64, device=DEV, dtype=torch.float64) / 64)).float()
    dots = []
    for base in (0, 1000, 1 << 20, (1 << 30) + 12345):
        a, _ = nf4.rope(q, k, torch.tensor([[base + 37]], dtype=torch.int32, device=DEV), inv)
        _, b = nf4.rope(q, k, torch.tensor([[base]], dtype=torch.int32, device=DEV), inv)
        dots.append(float((a.double() * b.double()).sum()))
    bound = 2.0 ** -7 * float((q.double().norm() * k.double().norm()))
    assert max(dots) - min(dots) <= bound


# ---------------------------------------------------------------------------------------------
# Residual RMS norm
# ---------------------------------------------------------------------------------------------
@pytest.mark.parametrize("rows,width", [(1, 2048), (1, 8), (3, 72), (5, 5120), (400, 5120), (2, 8200), (700, 1024),
                                        (2, 32768), (2, 40000), (350, 16384), (0, 64)])
@pytest.mark.parametrize("residual", [True, False])
def test_rmsnorm(rows, width, residual):
    x, w = randn((rows, width), 1), (1 + 0.2 * torch.randn(width, generator=gen(2), device=DEV)).to(torch.bfloat16)
    r = randn((rows, width), 3, 4.0) if residual else None
    if rows > 2:
        x[1] = 0
        if residual:
            r[1] = 0
        x[2] *= 1e-4
    h32 = x.float() + r.float() if residual else x.float()
    eps = 1e-6
    ro, y = Guarded(x.shape, torch.bfloat16), Guarded(x.shape, torch.bfloat16)
    y8, sc = Guarded(x.shape, torch.float8_e4m3fn), Guarded((rows,), torch.float32)
    nf4.nf4_rmsnorm(x, w, eps, residual=r, residual_out=ro.t, y=y.t, y8=y8.t, y8_scales=sc.t)
    assert all(g.canaries_intact() for g in (ro, y, y8, sc))
    assert torch.equal(ro.t, h32.to(torch.bfloat16))
    h = h32.double()
    want = h / torch.sqrt((h * h).mean(-1, keepdim=True) + eps) * w.double()
    assert bool(((y.t.double() - want).abs() <= 2.0 ** -8 * want.abs()).all())
    s64 = want.abs().amax(-1) / 448 if rows else torch.zeros(0, dtype=torch.float64, device=DEV)
    assert bool(((sc.t.double() - s64).abs() <= 2.0 ** -20 * s64).all())
    got = y8.t.float().double() * sc.t.double()[:, None]
    step = torch.maximum(2.0 ** -4 * want.abs(), 2.0 ** -10 * s64[:, None])
    assert bool(((got - want).abs() <= step * (1 + 2.0 ** -10)).all())
    # one output at a time, in place
    a, b = x.clone(), None if r is None else r.clone()
    nf4.nf4_rmsnorm(a, w, eps, residual=b, residual_out=b, y=a)
    assert torch.equal(a, y.t) and (b is None or torch.equal(b, ro.t))
    one8, ones = torch.empty_like(y8.t), torch.empty_like(sc.t)
    nf4.nf4_rmsnorm(x, w, eps, residual=r, y8=one8, y8_scales=ones)
    assert torch.equal(one8.view(torch.uint8), y8.t.view(torch.uint8)) and torch.equal(ones, sc.t)


def test_rmsnorm_eps_counts_for_small_rows():
    x = randn((2, 512), 1, 1e-3)
    w = torch.ones(512, dtype=torch.bfloat16, device=DEV)
    y = nf4.rmsnorm(x, w, 1e-2)
    h = x.double()
    want = h / torch.sqrt((h * h).mean(-1, keepdim=True) + 1e-2)
    assert bool(((y.double() - want).abs() <= 2.0 ** -8 * want.abs()).all())
