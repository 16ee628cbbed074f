"""Long attention calls whose values mark their place, so that a lost, doubled or misplaced part shows; and the accuracy
of long sums of values around zero (GPU).

Marks: V's key j of n is one in dim (j D // n + turn) mod D, a turn for each sequence and kv head, and zero
elsewhere, so that output d is the softmax weight of one run of n / D keys.  These are sums of positive terms, and
every error of the arithmetic is relative to them:
  2^-8              the output's rounding to bf16
  2^-11             p times V's scale in fp16 (fp8, NF4); p in two bf16 parts: 2^-16
  2 A e             a logit off by A e moves p, and the sum of p, by as much; A = max_j scale sum_d |q_d k_jd|;
                    e = 6.3e-4 for NF4 (a table entry in fp16), 2^-16 else (fp32 sums)
  2^-12             the fp32 sums of p and of p v (2^12 terms a chain at most)
A part of n / 304 keys (as many parts as the GPU has half-SM workers) is at least D / 608 of one of these runs: each test
checks that leaving any such part out of the 64-bit result is beyond the bound.

Around zero: the norm of the error over all outputs is bounded by that of the outputs' own rounding, which is
measured, and by what each key's rounding, independent of the others', adds: c^2 sum (p v)^2, with c^2 = 2^-28 (bf16: p to
2^-16, fp32 sums), 2^-22 (fp8: p s in fp16) and 3 2^-22 (NF4: p s; V's table entries; K's, through logits whose
products have a norm of at most sqrt(head_dim) scale), and for NF4 the table's mean error, 2.5e-6 sum p |v|.  A sixteenth
is added for the measured part's chance.
"""
import pytest
import torch

import nf4_weight_only_gb300 as nf4
from gpu_util import DEV
from test_layer_ops_gpu import FORMATS, TABLE, gen, paged, randn, values64

pytestmark = pytest.mark.gpu
PARTS = 304


def places(table, b, n, page):
    j = torch.arange(n, device=DEV)
    return table[b].to(DEV)[j // page].long() * page + j % page


def filled(fmt, lengths, heads, page, dim, seed, value):
    """A cache of keys with a drift along their sequence, and of value(b, n) -> [n, heads, dim]; its page table."""
    need = sum(-(-n // page) for n in lengths)
    c = nf4.KVCache.empty(fmt, need, heads, page, dim, DEV)
    table = paged(lengths, page, need, max(1, -(-max(lengths) // page)), seed)
    for b, n in enumerate(lengths):
        if not n:
            continue
        k = torch.randn((n, heads, dim), generator=gen(seed + 100 * b + 1), device=DEV)
        k[..., :8] += 6 * torch.sin(torch.arange(n, device=DEV) * (7 * torch.pi / n))[:, None, None]
        nf4.nf4_kv_append(c, k.to(torch.bfloat16), value(b, n).to(torch.bfloat16), places(table, b, n, page))
    assert nf4.nf4_check_device_error() == 0
    return c, table


def weights64(c, q, at, heads, group):
    """Softmax weights [heads, group, n] and A [heads, group] of one sequence, in 64 bits."""
    keys = values64(c, "k").transpose(1, 2).reshape(-1, heads, c.head_dim)[at].transpose(0, 1)
    qq = q.double().view(heads, group, c.head_dim)
    scale = c.head_dim ** -0.5
    return (torch.softmax(qq @ keys.transpose(1, 2) * scale, -1),
            scale * (qq.abs() @ keys.abs().transpose(1, 2)).amax(-1))


def spread(low, high, batch):
    n = torch.randint(low, high, (batch,), generator=torch.Generator().manual_seed(batch)).tolist()
    n[batch // 2] = 0
    return n


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("lengths,heads,group,dim,page", [
    ([30011, 29997], 1, 8, 128, 32),     # one kv head: joins in two stages
    ([70001], 1, 3, 64, 64),
    ([120001], 8, 5, 64, 64),            # by line, 38 parts a segment
    ([40001], 2, 8, 128, 64),
    ([40001], 1, 16, 128, 16),           # two tiles of heads
    ([9973], 1, 33, 64, 64),             # three groups of heads
    ([20011], 2, 12, 256, 128),
    ([15013, 1, 700, 0, 15], 3, 4, 128, 48),
    (spread(90, 4000, 33), 4, 2, 64, 64),    # by line, segments found by block
    (spread(2000, 9000, 24), 8, 1, 128, 64),
    (spread(700, 1100, 70), 1, 2, 64, 64),
])
def test_every_part_counts(fmt, lengths, heads, group, dim, page):
    def marks(b, n):
        at = (torch.arange(n, device=DEV) * dim // n)[:, None] + 7 * torch.arange(heads, device=DEV) + 3 * b
        return torch.nn.functional.one_hot(at % dim, dim)

    c, table = filled(fmt, lengths, heads, page, dim, 5, marks)
    q = randn((len(lengths), heads * group, dim), 9, 0.5)
    n_dev = torch.tensor(lengths, dtype=torch.int32, device=DEV)
    out = nf4.attention_decode(c, q, table.to(DEV), n_dev, nf4.attention_workspace(c, len(lengths), heads * group))
    assert nf4.nf4_check_device_error() == 0
    for b, n in enumerate(lengths):
        got = out[b].double().view(heads, group, dim)
        if n == 0:
            assert not got.any()
            continue
        p, big = weights64(c, q[b], places(table, b, n, page), heads, group)
        j = torch.arange(n, device=DEV)
        parts = max(1, min(PARTS, n // 256))
        mass = torch.zeros((heads, group, parts * dim), dtype=torch.float64, device=DEV)
        mass.index_add_(2, (j * parts // n) * dim + j * dim // n, p)
        mass = mass.view(heads, group, parts, dim)  # weight of each part in each run of n / dim keys
        want = mass.sum(2)
        relative = 2.0 ** -8 + 2.0 ** -12 + (0 if fmt == "bf16" else 2.0 ** -11)
        relative = relative + 2 * big * (6.3e-4 if fmt == "nf4" else 2.0 ** -16)
        tol = relative[..., None] * want + 2.0 ** -24
        for h in range(heads):  # dim (run + 7 h + 3 b) holds the run
            turned = torch.roll(got[h], -(7 * h + 3 * b), -1)
            assert bool(((turned - want[h]).abs() <= tol[h]).all())
        if parts > 1:
            left = (want[:, :, None] - mass) / (1 - mass.sum(-1, keepdim=True))
            assert bool((((left - want[:, :, None]).abs() / tol[:, :, None]).amax(-1) > 2).all())


def test_as_many_parts_as_workers():
    """The bound's PARTS is at least what this GPU's workers can make of one segment."""
    assert torch.cuda.get_device_properties(0).multi_processor_count * 2 <= PARTS


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("n,heads,group,dim", [(131071, 4, 5, 128), (60013, 2, 12, 64), (30011, 2, 4, 256)])
def test_long_sums_around_zero(fmt, n, heads, group, dim):
    page = 64
    need = -(-n // page)
    c = nf4.KVCache.empty(fmt, need, heads, page, dim, DEV)
    table = paged([n], page, need, need, 15)
    at = places(table, 0, n, page)
    nf4.nf4_kv_append(c, randn((n, heads, dim), 16), randn((n, heads, dim), 17), at)
    q = randn((1, heads * group, dim), 18)
    lengths = torch.tensor([n], dtype=torch.int32, device=DEV)
    out = nf4.attention_decode(c, q, table.to(DEV), lengths, nf4.attention_workspace(c, 1, heads * group))
    p, _ = weights64(c, q[0], at, heads, group)
    v = values64(c, "v").transpose(1, 2).reshape(-1, heads, dim)[at].transpose(0, 1)
    want = p @ v
    err = float((out.double().view(want.shape) - want).norm())
    own = float((want.to(torch.bfloat16).double() - want).norm())
    squares, sizes = float(((p * p) @ (v * v)).sum()), float((p @ v.abs()).norm())
    c2 = {"bf16": 2.0 ** -28, "fp8": 2.0 ** -22, "nf4": 3 * 2.0 ** -22}[fmt]
    bound = (own ** 2 + c2 * squares + ((2.5e-6 * sizes) ** 2 if fmt == "nf4" else 0)) ** 0.5 * (1 + 1 / 16)
    assert err <= bound
    # what the bound is there to see, planted in the 64-bit form
    if fmt == "bf16":  # weights in one bf16 part
        top = p.amax(-1, keepdim=True)
        planted = ((p / top).to(torch.bfloat16).double() * top) @ v
        assert float((planted.to(torch.bfloat16).double() - want).norm()) > bound
    if fmt == "nf4" and n > 100000:  # a table rounded entry by entry
        ratio = torch.tensor(TABLE, device=DEV).to(torch.float16).double() / torch.tensor(TABLE, dtype=torch.float64, device=DEV)
        codes = c.v.transpose(1, 2).reshape(-1, heads, dim // 2)[at].transpose(0, 1)
        f = torch.nan_to_num(ratio, nan=1.0)
        planted = p @ (v * torch.stack((f[(codes & 15).long()], f[(codes >> 4).long()]), -1).flatten(-2))
        assert float((planted - want).norm()) > bound
