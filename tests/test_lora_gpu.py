"""Low-rank adapters of many requests (nf4_lora_plan, nf4_lora) against 64-bit products (GPU).

Bound of y = bf16(base + s B h), h = A x: the last rounding is off by 2^-8 |y| at most.  A sum of n terms in fp32, each
addition off by 2^-23 of the sum so far (tensor-core sums may be cut, not rounded), is off by n 2^-23 of the sum of
the terms' sizes: n is at most K / 8 + 64 in the first product (a warp's steps of 16, then the warps, then the slices)
and rank + 64 in the second, and s h enters that as two bf16 numbers, off by 2^-16."""
import pytest
import torch

import nf4_weight_only_gb300 as nf4

from gpu_util import DEV, Guarded

pytestmark = pytest.mark.gpu


def bf(shape, g, scale=1.0):
    return (torch.randn(shape, generator=g, device=DEV) * scale).to(torch.bfloat16)


class Case:
    def __init__(self, t, k, ns, rank, adapters, ids, seed=0, in_place=False):
        g = torch.Generator(device=DEV).manual_seed(seed)
        self.t, self.k, self.ns, self.rank, self.adapters = t, k, ns, rank, adapters
        self.ids = torch.tensor(ids, dtype=torch.int32, device=DEV)
        self.x = bf((t, k), g)
        self.a = [bf((adapters, rank, k), g, k ** -0.5) for _ in ns]
        self.b = [bf((adapters, n, rank), g) for n in ns]
        self.scales = torch.rand(adapters, generator=g, device=DEV) * 3 - 1
        self.base = [bf((t, n), g) for n in ns]
        self.ys = [Guarded((t, n), torch.bfloat16) for n in ns]
        self.in_place = in_place
        for y, base in zip(self.ys, self.base):
            y.t.copy_(base if in_place else torch.full_like(base, float("nan")))
        self.plan = nf4.lora_plan(self.ids, adapters)
        self.workspace = nf4.lora_workspace(t, adapters, rank, len(ns))
        self.workspace.fill_(0xFF)  # needs no set-up

    def run(self, stream=None):
        nf4.nf4_lora(self.x, self.plan, self.scales, self.a, self.b, [y.t for y in self.ys], self.workspace,
                     bases=None if self.in_place else self.base, stream=stream)

    def check(self, sample=None):
        rows = range(self.t) if sample is None else sample
        lists = {}
        for r in rows:
            lists.setdefault(int(self.ids[r]), []).append(r)
        for y, a, b, base in zip(self.ys, self.a, self.b, self.base):
            assert y.canaries_intact()
            for adapter, at in lists.items():
                at = torch.tensor(at, device=DEV)
                got = y.t[at]
                if adapter < 0:
                    assert torch.equal(got, base[at])
                    continue
                x, aa, bb = self.x[at].double(), a[adapter].double(), b[adapter].double()
                s = float(self.scales[adapter])
                h = x @ aa.T
                want = base[at].double() + s * (h @ bb.T)
                size = x.abs() @ aa.abs().T
                first, second = (self.k / 8 + 64) * 2.0 ** -23, (self.rank + 64) * 2.0 ** -23 + 2.0 ** -16
                bound = 2.0 ** -8 * want.abs() + abs(s) * ((size * first + h.abs() * second) @ bb.abs().T) * 1.01 + \
                    2.0 ** -22 * base[at].double().abs() + 1e-30
                assert bool(((got.double() - want).abs() <= bound).all())
        assert nf4.nf4_check_device_error() == 0


def spread(t, adapters, seed, idle=0.1):
    g = torch.Generator().manual_seed(seed)
    ids = torch.randint(0, adapters, (t,), generator=g)
    ids[torch.rand(t, generator=g) < idle] = -1
    return ids.tolist()


@pytest.mark.parametrize("t", [1, 2, 7, 16, 17, 33, 64, 65, 130, 515])
@pytest.mark.parametrize("rank", [8, 16, 24, 64, 128])
def test_token_counts_and_ranks(t, rank):
    c = Case(t, 512, [64, 24], rank, 3, spread(t, 3, t + rank), seed=t + rank)
    c.run()
    c.check()


@pytest.mark.parametrize("k", [64, 128, 192, 320, 2048, 5120, 13824, 27648])
@pytest.mark.parametrize("t", [1, 40])
def test_widths(k, t):
    c = Case(t, k, [40], 16, 2, spread(t, 2, k, idle=0), seed=k)
    c.run()
    c.check()


@pytest.mark.parametrize("ns", [[1], [2], [7], [8], [31], [257], [263, 1, 40], [264], [1000, 16], [8, 8, 8, 8, 8, 8, 8, 8],
                                [0, 24, 0]])
@pytest.mark.parametrize("in_place", [False, True])
def test_heights_and_groups(ns, in_place):
    """Odd heights (rows of y that start anywhere), up to eight projections, empty ones among them."""
    c = Case(37, 256, ns, 16, 4, spread(37, 4, 5), seed=sum(ns), in_place=in_place)
    c.run()
    c.check()


@pytest.mark.parametrize("kind", ["none", "all one", "each its own", "runs", "last", "one of many"])
@pytest.mark.parametrize("in_place", [False, True])
def test_who_has_which_adapter(kind, in_place):
    t, adapters = 150, 200
    ids = {"none": [-1] * t, "all one": [7] * t, "each its own": list(range(t)), "runs": [i // 70 for i in range(t)],
           "last": [-1] * (t - 1) + [adapters - 1], "one of many": [3] + [-5] * (t - 1)}[kind]
    c = Case(t, 192, [48, 16], 32, adapters, ids, in_place=in_place)
    c.run()
    c.check()


def test_no_adapters_loaded():
    t = 5
    base = [torch.randn((t, 16), device=DEV).to(torch.bfloat16)]
    y = [torch.zeros_like(base[0])]
    x = torch.zeros((t, 64), dtype=torch.bfloat16, device=DEV)
    plan = nf4.lora_plan(torch.full((t,), -1, dtype=torch.int32, device=DEV), 0)
    none = torch.zeros((0, 8, 64), dtype=torch.bfloat16, device=DEV), torch.zeros((0, 16, 8), dtype=torch.bfloat16, device=DEV)
    nf4.nf4_lora(x, plan, torch.zeros(0, device=DEV), [none[0]], [none[1]], y, nf4.lora_workspace(t, 0, 8, 1), bases=base)
    assert torch.equal(y[0], base[0]) and nf4.nf4_check_device_error() == 0


def test_a_row_does_not_see_its_neighbours():
    """A token's result is the same bytes alone, in a batch, and beside a token of NaN and infinities."""
    c = Case(90, 640, [72], 16, 3, spread(90, 3, 1, idle=0), seed=4)
    c.run()
    first = c.ys[0].t.clone()
    c.x[11] = float("nan")
    c.x[55] = float("inf")
    c.ys[0].t.zero_()
    c.run()
    keep = [r for r in range(90) if r not in (11, 55)]
    assert torch.equal(c.ys[0].t[keep], first[keep])
    order = torch.randperm(90, generator=torch.Generator().manual_seed(3)).to(DEV)
    d = Case(90, 640, [72], 16, 3, c.ids[order].tolist(), seed=4)
    d.x.copy_(torch.where(torch.isfinite(c.x), c.x, 0)[order])
    d.base[0].copy_(c.base[0][order])
    d.run()
    clean = ~((order == 11) | (order == 55))
    assert torch.equal(d.ys[0].t[clean], first[order][clean])


def test_prompts_and_a_high_rank():
    ids = [i // 700 % 4 - 1 for i in range(3001)]
    c = Case(3001, 1024, [520, 136], 64, 3, ids, seed=9)
    c.run()
    c.check()
    c = Case(5000, 256, [64], 16, 5, [i // 1100 for i in range(5000)], seed=10)
    c.run()
    c.check()


def test_many_adapters_and_tokens():
    """8192 loaded adapters, and more tokens than a round of the plan takes."""
    c = Case(2500, 64, [16], 8, 8192, [(i * 37) % 8192 for i in range(2500)], seed=2)
    c.run()
    c.check(range(0, 2500, 25))


def plan_lists(plan, t, adapters):
    words = plan.view(torch.int32).tolist()
    assert words[:2] == [t, adapters]
    many, few, n_tokens = words[2:5]
    chunks = [words[8 + 4 * i:11 + 4 * i] for i in range(many + few)]
    assert all(n > 16 for _, _, n in chunks[:many]) and all(n <= 16 for _, _, n in chunks[many:])
    order = words[len(words) - t:]
    return chunks, order, n_tokens


@pytest.mark.parametrize("t,adapters", [(0, 3), (1, 1), (63, 2), (64, 1), (65, 1), (300, 7), (1024, 300), (5000, 3),
                                        (5000, 2000), (70000, 40)])
@pytest.mark.parametrize("layout", ["mixed", "runs"])
def test_plan(t, adapters, layout):
    ids = spread(t, adapters, t, idle=0.2) if layout == "mixed" else [i * adapters // max(1, t) for i in range(t)]
    ids_t = torch.tensor(ids, dtype=torch.int32, device=DEV)
    plan = nf4.lora_plan(ids_t, adapters)
    chunks, order, n_tokens = plan_lists(plan, t, adapters)
    want = sorted(range(t), key=lambda i: (ids[i] < 0, ids[i]))  # stable
    assert order == want and n_tokens == sum(i >= 0 for i in ids)
    at = 0
    for adapter, first, n in sorted(chunks, key=lambda c: c[1]):
        assert first == at and 1 <= n <= 64
        assert all(ids[i] == adapter for i in order[first:first + n])
        at += n
        assert at == n_tokens or n == 64 or ids[order[at]] != adapter
    assert at == n_tokens
    again = nf4.lora_plan(ids_t, adapters)
    used = 16 * (2 + len(chunks))
    assert torch.equal(plan[:used], again[:used]) and nf4.nf4_check_device_error() == 0


def test_plan_from_sequences():
    ids = torch.tensor([2, -1, 0, 1], dtype=torch.int32, device=DEV)
    sequences = torch.tensor([3, 3, 0, 1, -1, 2, 0, -1], dtype=torch.int32, device=DEV)
    chunks, order, n = plan_lists(nf4.lora_plan(ids, 3, sequences), 8, 3)
    assert chunks == [[0, 0, 1], [1, 1, 2], [2, 3, 2]] and order == [5, 0, 1, 2, 6, 3, 4, 7] and n == 5


def test_ids_outside_the_list_count_as_none():
    assert nf4.nf4_check_device_error() == 0
    ids = torch.tensor([0, 4, 3, 1 << 30], dtype=torch.int32, device=DEV)
    chunks, order, n = plan_lists(nf4.lora_plan(ids, 4), 4, 4)
    assert chunks == [[0, 0, 1], [3, 1, 1]] and order == [0, 2, 1, 3] and nf4.nf4_check_device_error() == 46
    sequences = torch.tensor([0, 4, 2, 1], dtype=torch.int32, device=DEV)
    ids = torch.tensor([1, 1, 1, 1], dtype=torch.int32, device=DEV)
    chunks, order, n = plan_lists(nf4.lora_plan(ids, 2, sequences), 4, 2)
    assert chunks == [[1, 0, 3]] and order == [0, 2, 3, 1] and nf4.nf4_check_device_error() == 46


def test_a_plan_of_other_sizes_is_reported():
    c = Case(20, 128, [16], 8, 3, spread(20, 3, 1))
    assert nf4.nf4_check_device_error() == 0
    for other in (nf4.lora_plan(c.ids[:19], 3), nf4.lora_plan(c.ids, 4), torch.zeros_like(c.plan),
                  torch.full_like(c.plan, 0x7F)):
        c.plan = torch.cat((other, torch.zeros(4096, dtype=torch.uint8, device=DEV)))
        c.ys[0].t.fill_(3.0)
        c.run()
        assert nf4.nf4_check_device_error() == 47
        assert bool((c.ys[0].t == 3.0).all()) and c.ys[0].canaries_intact()


def test_captured_repeated_and_on_streams():
    cases = [Case(120, 1024, [264, 64], 16, 5, spread(120, 5, i), seed=i) for i in range(3)]
    for c in cases:
        c.run()
        c.want = [y.t.clone() for y in c.ys]
    streams = [torch.cuda.Stream() for _ in cases]
    torch.cuda.synchronize()
    for _ in range(5):
        for c, s in zip(cases, streams):
            c.run(s)
    torch.cuda.synchronize()
    for c in cases:
        assert all(torch.equal(y.t, w) for y, w in zip(c.ys, c.want))
    c = cases[0]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        nf4.nf4_lora_plan(c.ids, c.adapters, c.plan)
        c.run()
    for y in c.ys:
        y.t.zero_()
    graph.replay()
    assert all(torch.equal(y.t, w) for y, w in zip(c.ys, c.want))
    c.ids.copy_(torch.tensor(spread(120, 5, 77), dtype=torch.int32))
    graph.replay()
    c.check()


def test_one_workspace_serves_smaller_calls():
    big = Case(300, 2048, [64], 16, 4, spread(300, 4, 1), seed=1)
    for t in (1, 50, 200):
        c = Case(t, 2048, [64], 16, 4, spread(t, 4, t, idle=0), seed=t)
        c.workspace = big.workspace
        c.run()
        big.run()
        c.check()
        big.check()


@pytest.mark.parametrize("ns,in_place", [([520, 136], True), ([256], False), ([8], True), ([24, 1000], False), ([57, 64], True)])
@pytest.mark.parametrize("rank", [8, 16, 32, 64, 128])
def test_long_prompts(ns, in_place, rank):
    """Calls with many tokens: rows that 16-byte copies reach and rows that they do not, last blocks of eight columns,
    chunks of 64 and of less beside rows without an adapter."""
    t = 1700
    ids = ([0] * 700 + [-1] * 61 + [2] * 337 + [1] * 90 + [2] * 64 + [4] * 5 + [0] * 300)
    ids += [-1] * (t - len(ids))
    c = Case(t, 320, ns, rank, 5, ids, seed=rank + len(ns), in_place=in_place)
    c.run()
    first = [y.t.clone() for y in c.ys]
    c.check()
    if not in_place:
        c.run()
        assert all(torch.equal(y.t, f) for y, f in zip(c.ys, first))


@pytest.mark.parametrize("t", [5, 40])
@pytest.mark.parametrize("rank", [8, 16, 64])
def test_infinities(t, rank):
    """An infinite input, and products past the range of fp32, give what they give in the formula, in their row alone."""
    c = Case(t, 128, [40], rank, 1, [0] * t, seed=t)
    c.a[0].zero_()
    c.a[0][0, :, 3] = 1.0  # h_r = x[3], and y = base + s x[3] (the sum of B's row)
    c.b[0].copy_(c.b[0].abs() + 1)
    c.b[0][0, 1::2] *= -1
    c.scales.fill_(0.5)
    for row, value in [(0, float("inf")), (t - 1, -float("inf")), (2, float("nan"))]:
        c.x[row, 3] = value
    c.run()
    y = c.ys[0].t.float()
    up = torch.tensor([1.0, -1.0] * 20, device=DEV) * float("inf")
    assert torch.equal(y[0], up) and torch.equal(y[t - 1], -up) and bool(y[2].isnan().all())
    keep = [r for r in range(t) if r not in (0, 2, t - 1)]
    assert bool(y[keep].isfinite().all())
    c.check(sample=keep)


@pytest.mark.parametrize("ns", [[57, 320], [1, 259], [41]])
@pytest.mark.parametrize("rank,in_place", [(16, False), (24, True), (64, False), (128, True), (128, False)])
def test_rows_that_begin_anywhere(ns, rank, in_place):
    """Odd heights with chunks of 64, of less and of few, and whole and broken runs of rows without an adapter."""
    ids = [-1] * 71 + [0] * 150 + [-1] * 9 + [1] * 13 + [2] * 64 + [3] + [-1] * 64
    c = Case(len(ids), 192, ns, rank, 4, ids, seed=rank + len(ns), in_place=in_place)
    c.run()
    c.check()
