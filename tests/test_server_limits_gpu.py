"""The operators of a server at the largest sizes that they take (GPU), and calls that mix what others have apart."""
import pytest
import torch

import nf4_weight_only_gb300 as nf4

from gpu_util import DEV, Guarded
from test_lora_gpu import Case, spread

pytestmark = pytest.mark.gpu


def enough(gigabytes):
    torch.cuda.empty_cache()
    if torch.cuda.mem_get_info()[0] < gigabytes << 30:
        pytest.skip(f"needs {gigabytes} GB of device memory")


def test_plan_of_the_most_rows():
    """2^31 - 1 rows: two prompts that fill all but nine of them, a sequence of one token and one that no longer fits."""
    enough(48)
    t, page, half = (1 << 31) - 1, 65536, (1 << 30) - 5
    i32, i64 = torch.int32, torch.int64
    lengths = torch.tensor([0, 3, 65536, 7], dtype=i32, device=DEV)
    new = torch.tensor([half, half, 1, 12], dtype=i32, device=DEV)
    table = torch.zeros((4, 16385), dtype=i32, device=DEV)
    table[1, 0], table[2, 0], table[3, 0] = 40000, 40001, 40002
    ring, state = nf4.free_ring(50000)
    state.copy_(torch.tensor([1000, 39000]))
    out = torch.zeros(4, dtype=i32, device=DEV)
    starts = torch.zeros(5, dtype=i32, device=DEV)
    slots = torch.full((t,), -7, dtype=i64, device=DEV)
    positions, sequences = (torch.full((t,), -7, dtype=i32, device=DEV) for _ in range(2))
    nf4.nf4_plan_step(lengths, new, page, table, ring, state, state, out, starts, slots, positions, sequences)
    assert starts.tolist() == [0, half, 2 * half, 2 * half + 1, t]  # (sums stop there)
    assert out.tolist() == [half, half + 3, 65537, 7]
    held = [0, 1, 1, 1]
    first = 1000
    for b, n in enumerate([half, half, 1]):
        need = -(-(int(lengths[b]) + n) // page) - held[b]
        assert torch.equal(table[b, held[b]:held[b] + need], torch.arange(first, first + need, dtype=i32, device=DEV))
        first += need
    assert state.tolist() == [first, 40000 - first]
    chunk = 1 << 27
    for b, (at, n) in enumerate([(0, half), (half, half), (2 * half, 1)]):
        for i in range(0, n, chunk):
            m = min(chunk, n - i)
            pos = torch.arange(i, i + m, device=DEV) + int(lengths[b])
            assert torch.equal(positions[at + i:at + i + m], pos.to(i32))
            assert bool((sequences[at + i:at + i + m] == b).all())
            assert torch.equal(slots[at + i:at + i + m], table[b, pos // page].long() * page + pos % page)
    rest = slice(2 * half + 1, t)
    assert bool((slots[rest] == -1).all()) and bool((sequences[rest] == 3).all())
    assert positions[rest].tolist() == [7 + i for i in range(t - 2 * half - 1)]
    assert nf4.nf4_check_device_error() == 0
    del slots, positions, sequences
    torch.cuda.empty_cache()


def test_adapters_of_the_most_tokens():
    """2^24 tokens of 8192 loaded adapters: one with most of them, many with a few, some with none."""
    enough(16)
    t, adapters = 1 << 24, 8192
    g = torch.Generator(device=DEV).manual_seed(1)
    ids = torch.full((t,), 8191, dtype=torch.int32, device=DEV)
    few = torch.randint(0, t, (90000,), generator=g, device=DEV)
    ids[few] = torch.randint(-1, 5000, (90000,), generator=g, device=DEV).to(torch.int32)
    bf = torch.bfloat16
    x = torch.empty((t, 64), dtype=bf, device=DEV).normal_(generator=g)
    a = (torch.randn((adapters, 8, 64), generator=g, device=DEV) / 8).to(bf)
    b = torch.randn((adapters, 8, 8), generator=g, device=DEV).to(bf)
    scales = torch.rand(adapters, generator=g, device=DEV) + 0.5
    base = torch.empty((t, 8), dtype=bf, device=DEV).normal_(generator=g)
    y = Guarded((t, 8), bf)
    plan = nf4.lora_plan(ids, adapters)
    nf4.nf4_lora(x, plan, scales, [a], [b], [y.t], nf4.lora_workspace(t, adapters, 8, 1), bases=[base])
    assert nf4.nf4_check_device_error() == 0 and y.canaries_intact()
    assert torch.equal(plan.view(torch.int32)[-t:].long().sort().values, torch.arange(t, device=DEV))
    ask = torch.cat((few, torch.arange(0, t, 997, device=DEV), torch.arange(t - 100, t, device=DEV)))
    for at in ask.split(20000):
        i = ids[at].long().clamp_min(0)
        s = torch.where(ids[at] >= 0, scales[i], 0.0).double()[:, None]
        aa, bb, xx = a[i].double(), b[i].double(), x[at].double()
        h, size = torch.einsum("trk,tk->tr", aa, xx), torch.einsum("trk,tk->tr", aa.abs(), xx.abs())
        want = base[at].double() + s * torch.einsum("tnr,tr->tn", bb, h)
        # as in test_lora_gpu.py: K / 8 + 64 and rank + 64 additions, two bf16 numbers, the last rounding
        off = size * 72 * 2.0 ** -23 + h.abs() * (72 * 2.0 ** -23 + 2.0 ** -16)
        bound = 2.0 ** -8 * want.abs() + s * torch.einsum("tnr,tr->tn", bb.abs(), off) * 1.01 + \
            2.0 ** -22 * base[at].double().abs()
        assert bool(((y.t[at].double() - want).abs() <= bound).all())


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_samples_of_the_most_rows(dtype):
    """2^24 rows of three logits, one of them masked: u below the first one's share draws it, else the last."""
    enough(8)
    b = 1 << 24
    g = torch.Generator(device=DEV).manual_seed(2)
    l = torch.zeros((b, 3), dtype=dtype, device=DEV)
    l[:, 1] = -float("inf")
    u = torch.rand(b, generator=g, device=DEV)
    tokens = Guarded((b,), torch.int32)
    nf4.nf4_sample(l, u, tokens.t)
    assert torch.equal(tokens.t, (u >= 0.5).int() * 2) and tokens.canaries_intact()
    assert nf4.nf4_check_device_error() == 0


def test_some_projections_in_place():
    """Of three projections one has a base of its own; two have the same A and the same base."""
    t = 230
    c = Case(t, 320, [72, 41, 72], 16, 4, spread(t, 4, 5), seed=8)
    c.a[2], c.base[2] = c.a[0], c.base[0]
    c.ys[1].t.copy_(c.base[1])
    bases = [c.base[0], c.ys[1].t, c.base[2]]
    nf4.nf4_lora(c.x, c.plan, c.scales, c.a, c.b, [y.t for y in c.ys], c.workspace, bases=bases)
    c.check()


@pytest.mark.parametrize("lengths_in_place,state_in_place", [(True, False), (False, True), (True, True)])
def test_plans_partly_in_place(lengths_in_place, state_in_place):
    import numpy as np
    from test_plan_step_gpu import make
    rng = np.random.default_rng(12)
    s = make(rng, 700, 16, 12, 9000, finished=0.1, idle=0.1, long=0.4, spare=900)
    if lengths_in_place:
        s.lengths_out = s.lengths
    if state_in_place:
        s.state_out = s.state
    s.run()
    s.check()
    assert nf4.nf4_check_device_error() == 0
