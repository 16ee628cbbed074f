"""The attention's ways of cutting its work, each at sizes that reach it (GPU): results against 64 bits, the
same bytes on every call, and a workspace that serves all of them in turn."""
import pytest
import torch

import nf4_weight_only_gb300 as nf4
from gpu_util import DEV
from test_layer_ops_gpu import FORMATS, new_cache, paged, randn, reference

pytestmark = pytest.mark.gpu


def lengths_of(kind, batch):
    g = torch.Generator().manual_seed(batch)
    if kind == "equal":
        return [1723] * batch
    if kind == "ragged":
        return torch.randint(0, 2500, (batch,), generator=g).tolist()
    if kind == "short":
        return torch.randint(0, 60, (batch,), generator=g).tolist()
    if kind == "outlier":  # many short sequences and two long ones
        n = torch.randint(1, 40, (batch,), generator=g).tolist()
        n[batch // 3], n[-1] = 9001, 6000
        return n
    return [int(kind)] * batch


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("kind,batch,heads,group,dim", [
    ("equal", 24, 8, 1, 64),     # more segments than half the workers: equal runs (nf4) or tickets
    ("ragged", 40, 8, 2, 64),    # the same, ragged, more than 32 sequences
    ("short", 700, 2, 4, 128),   # workers of one warp, some of which write their output alone
    ("outlier", 700, 2, 2, 64),  # the same with pieces of long segments
    ("short", 2100, 1, 2, 64),   # more sequences than are found by block
    ("short", 4200, 1, 1, 64),   # more than are kept while the plan is made
    ("30011", 2, 1, 8, 128),     # one kv head: joins in two stages
    ("70001", 1, 1, 3, 64),
])
def test_cuts(fmt, kind, batch, heads, group, dim):
    lengths, page = lengths_of(kind, batch), 32
    need = sum(-(-n // page) for n in lengths)
    c = new_cache(fmt, need, heads, page, dim, seed=7)
    table = paged(lengths, page, need, -(-max(lengths) // page), 8)
    q = randn((batch, heads * group, dim), 9)
    n = torch.tensor(lengths, dtype=torch.int32, device=DEV)
    ws = nf4.attention_workspace(c, batch, heads * group)
    first = nf4.attention_decode(c, q, table.to(DEV), n, ws)
    for _ in range(4):
        assert torch.equal(nf4.attention_decode(c, q, table.to(DEV), n, ws), first)
    assert nf4.nf4_check_device_error() == 0
    control = ws[:16].view(torch.int32)
    assert not control.any()  # the tickets are as they were found
    # 64 bits: every sequence of the smaller batches, a spread of the others
    some = list(range(batch)) if batch <= 40 else sorted({0, 1, batch // 3, batch // 2, batch - 2, batch - 1}
                                                         | set(range(0, batch, batch // 50)))
    want, tol = reference(c, q[some], table[some], [lengths[i] for i in some], dim ** -0.5, 0)
    assert bool(((first[some].double() - want).abs() <= tol).all())
    empty = [i for i, m in enumerate(lengths) if m == 0]
    assert not first[empty].any()


def test_one_workspace_for_every_cut():
    """Calls that are cut in different ways, one after another on one workspace."""
    cases = []
    for fmt, kind, batch, heads, group in (("nf4", "equal", 24, 8, 1), ("bf16", "short", 700, 2, 4), ("fp8", "30011", 1, 1, 8),
                                           ("nf4", "ragged", 9, 4, 4), ("bf16", "equal", 24, 8, 1)):
        lengths, page = lengths_of(kind, batch), 64
        need = sum(-(-n // page) for n in lengths)
        c = new_cache(fmt, need, heads, page, 64, seed=17)
        table = paged(lengths, page, need, -(-max(lengths) // page), 18).to(DEV)
        q = randn((batch, heads * group, 64), 19)
        cases.append((c, q, table, torch.tensor(lengths, dtype=torch.int32, device=DEV)))
    own = [nf4.attention_decode(c, q, t, n, nf4.attention_workspace(c, *q.shape[:2])) for c, q, t, n in cases]
    size = max(nf4.nf4_attention_workspace_bytes(c, *q.shape[:2]) for c, q, _, _ in cases)
    shared = torch.zeros(size, dtype=torch.uint8, device=DEV)
    for _ in range(3):
        for (c, q, t, n), want in zip(cases, own):
            assert torch.equal(nf4.attention_decode(c, q, t, n, shared), want)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("batch,heads,group,low,high", [
    (1, 8, 5, 120001, 120002),   # few segments, long
    (33, 4, 2, 1, 9000),         # found by block
    (64, 8, 1, 90, 4000),        # cells of one long segment's part, and of many short segments
    (2100, 1, 2, 700, 1100),     # more sequences than are found by block
    (4200, 1, 1, 800, 1000),     # more than are kept while the plan is made
])
def test_line(fmt, batch, heads, group, low, high):
    """Segments laid end to end, some of them empty, with cells that end anywhere in them."""
    page, dim = 64, 64
    lengths = torch.randint(low, high, (batch,), generator=torch.Generator().manual_seed(batch)).tolist()
    for i in range(5, batch, 11):
        lengths[i] = 0
    need = sum(-(-n // page) for n in lengths)
    c = new_cache(fmt, need, heads, page, dim, seed=27)
    table = paged(lengths, page, need, -(-max(lengths) // page), 28)
    q = randn((batch, heads * group, dim), 29)
    n = torch.tensor(lengths, dtype=torch.int32, device=DEV)
    ws = nf4.attention_workspace(c, batch, heads * group)
    first = nf4.attention_decode(c, q, table.to(DEV), n, ws)
    assert torch.equal(nf4.attention_decode(c, q, table.to(DEV), n, ws), first)
    assert nf4.nf4_check_device_error() == 0
    some = sorted(set(range(0, batch, max(1, batch // 60))) | {batch - 1})
    want, tol = reference(c, q[some], table[some], [lengths[i] for i in some], dim ** -0.5, 0)
    assert bool(((first[some].double() - want).abs() <= tol).all())
    assert not first[[i for i, m in enumerate(lengths) if m == 0]].any()
