"""nf4_lora_plan and nf4_lora in buffers of exactly the bytes that they ask for, between guard bands (GPU), and products past
the range of fp32."""
import pytest
import torch

import nf4_weight_only_gb300 as nf4

from gpu_util import DEV, Guarded
from test_lora_gpu import Case

pytestmark = pytest.mark.gpu


def runs(*lengths):
    """Adapter 0 for so many tokens, then adapter 1, ...; negative: tokens without an adapter."""
    ids = []
    for i, n in enumerate(lengths):
        ids += [i if n > 0 else -1] * abs(n)
    return ids


# as many chunks of many (17 tokens) and of few as the sizes allow, as many slices of K as there are, ranks and counts at their ends
CASES = [
    (64, [8], 8, runs(1)),
    (27648, [8], 128, runs(1)),
    (27648, [8, 8, 8, 8, 8, 8, 8, 8], 128, runs(1, 2, 3)),
    (16384, [40, 8], 16, runs(17)),
    (16384, [40], 64, runs(17, 17)),
    (8192, [24], 8, runs(*[17] * 20)),
    (512, [24], 8, runs(*[17] * 310)),
    (512, [8] * 8, 128, runs(*[17] * 40, *[16] * 7)),
    (1024, [8], 16, runs(*[1] * 303)),
    (1024, [8], 16, runs(*[1] * 304)),
    (1024, [8], 16, runs(*[1] * 305)),
    (256, [64], 32, runs(*[16] * 100)),
    (8192, [16], 24, runs(64 * 5 + 1, -30, 64 * 3 + 17, 16)),
    (576, [16, 16], 40, runs(1000, 999, 998, -1)),
]


@pytest.mark.parametrize("case", range(len(CASES)))
def test_buffers_of_the_bytes_asked_for(case):
    k, ns, rank, ids = CASES[case]
    adapters = max(ids) + 1
    c = Case(len(ids), k, ns, rank, adapters, ids, seed=case)
    plan = Guarded((nf4.nf4_lora_plan_bytes(len(ids), adapters),), torch.uint8)
    workspace = Guarded((nf4.nf4_lora_workspace_bytes(len(ids), adapters, rank, len(ns)),), torch.uint8)
    plan.t.fill_(0x7F)
    workspace.t.fill_(0xFF)
    nf4.nf4_lora_plan(c.ids, adapters, plan.t)
    assert plan.canaries_intact() and torch.equal(plan.t[:20], c.plan[:20])
    before = plan.t.clone()
    c.plan, c.workspace = plan.t, workspace.t
    c.run()
    c.check()
    assert workspace.canaries_intact() and plan.canaries_intact() and torch.equal(plan.t, before)


@pytest.mark.parametrize("t", [5, 40])
@pytest.mark.parametrize("rank", [8, 24, 128])
@pytest.mark.parametrize("x,scale", [(3.0e38, 4.0),    # s h past the range
                                     (3.38e38, 0.5)])  # h past it, of two such inputs
def test_products_past_the_range(t, rank, x, scale):
    """Finite inputs: A takes x[3] + x[4], B's rows are 1 or more, or -1 or less, so every y of the row is past the range."""
    c = Case(t, 128, [40], rank, 1, [0] * t, seed=t)
    c.a[0].zero_()
    c.a[0][0, :, 3:5] = 1.0
    c.b[0].copy_(c.b[0].abs() + 1)
    c.b[0][0, 1::2] *= -1
    c.scales.fill_(scale)
    c.x[:, 3:5] = 0.25
    c.x[1, 3:5] = torch.tensor([x, 0.0 if scale > 1 else x], device=DEV)
    c.x[3, 3:5] = -c.x[1, 3:5]
    assert bool(c.x.isfinite().all())
    c.run()
    y = c.ys[0].t.float()
    up = torch.tensor([1.0, -1.0] * 20, device=DEV) * float("inf")
    assert torch.equal(y[1], up) and torch.equal(y[3], -up)
    c.check(sample=[r for r in range(t) if r not in (1, 3)])
