"""The choice of the next token (nf4_sample) against its definition in 64 bits (GPU).  Tokens are equal or wrong; a
token whose border lies within 1e-9 of the random number (in shares of the whole) is not asked about, and the inputs
are such that there is none.  logprobs: the sum of exp over V values in fp32 pieces is within 2^-20 of itself (each
exp2f is within 2 ulp, its argument within 2^-24 * 30 / ln 2 of the exact one, the pieces of a thread are below 600), so
log within 2^-20, and the result within 2^-22 of its size more."""
import numpy as np
import pytest
import torch

import nf4_weight_only_gb300 as nf4

from gpu_util import DEV, Guarded

pytestmark = pytest.mark.gpu


def definition(logits, u, temperature=1.0, k=0, p=1.0, least=0.0):
    """(token, logprob, distance of u from the nearest border in shares) of one row, float64 numpy."""
    l = np.asarray(logits, np.float64)
    real = ~(np.isnan(l) | (l == -np.inf))
    if not real.any():
        return -1, -np.inf, 1.0
    l = np.where(real, l, -np.inf)
    top = l.max()
    logs = l - top - np.log(np.exp(l - top).sum())
    if temperature == 0:
        token = int(np.argmax(l))
        return token, logs[token], 1.0
    w = np.exp((l - top) / temperature)
    order = np.lexsort((np.arange(len(l)), -l))
    order = order[real[order]]
    if 0 < k < len(order):
        order = order[:k]
    near = 1.0
    if p < 1:
        sums = np.cumsum(w[order])
        want = max(p, 0.0) * sums[-1]
        near = np.abs(sums - want).min() / sums[-1] if len(order) > 1 else 1.0
        order = order[:1 + np.count_nonzero(sums[:-1] < want)]
    order = order[w[order] >= min(max(least, 0.0), 1.0)]
    order = np.sort(order)
    sums = np.cumsum(w[order])
    at = int(np.searchsorted(sums, u * sums[-1], side="right"))
    near = min(near, np.abs(sums[:-1] / sums[-1] - u).min() if len(sums) > 1 else 1.0)
    token = int(order[min(at, len(order) - 1)])
    return token, logs[token], near


def call(logits, u, vocab=None, logprobs=True, **settings):
    b = logits.shape[0]
    tokens, logs = Guarded((b,), torch.int32), Guarded((b,), torch.float32)
    types = dict(temperature=torch.float32, top_k=torch.int32, top_p=torch.float32, min_p=torch.float32)
    given = {n: torch.tensor(v, dtype=types[n], device=DEV) for n, v in settings.items()}
    nf4.nf4_sample(logits, torch.tensor(u, dtype=torch.float32, device=DEV), tokens.t, vocab=vocab,
                   logprobs=logs.t if logprobs else None, **given)
    assert tokens.canaries_intact() and logs.canaries_intact()
    return tokens.t.tolist(), logs.t.tolist()


def compare(logits, u, vocab=None, **settings):
    b = logits.shape[0]
    tokens, logs = call(logits, u, vocab, **settings)
    host = logits.float().cpu().numpy()[:, :vocab]
    u = np.asarray(u, np.float32)
    asked = 0
    for i in range(b):
        row = {n: float(np.float32(v[i])) for n, v in settings.items()}
        want, log, near = definition(host[i], float(u[i]), row.get("temperature", 1.0), int(row.get("top_k", 0)),
                                     row.get("top_p", 1.0), row.get("min_p", 0.0))
        if near < 1e-9:
            continue
        asked += 1
        assert tokens[i] == want, (i, row, near)
        if want >= 0:
            assert abs(logs[i] - log) <= 2.0 ** -20 + 2.0 ** -22 * abs(log), (i, logs[i], log)
        else:
            assert logs[i] == -np.inf
    assert asked >= b - b // 16
    assert nf4.nf4_check_device_error() == 0


def rows(b, v, seed, dtype=torch.float32, spread=2.0, stride=None):
    g = torch.Generator(device=DEV).manual_seed(seed)
    l = torch.randn((b, stride or v), generator=g, device=DEV) * spread
    at = torch.randint(0, v, (b, 8), generator=g, device=DEV)
    l.scatter_add_(1, at, torch.rand((b, 8), generator=g, device=DEV) * 4 * spread)
    return l.to(dtype), torch.rand(b, generator=g, device=DEV).tolist()


SETTINGS = [dict(), dict(temperature=0.7), dict(top_k=1), dict(top_k=5), dict(top_k=50, top_p=0.9, temperature=0.8),
            dict(top_p=0.5), dict(top_p=0.99, min_p=0.01), dict(min_p=0.2), dict(min_p=1.0), dict(temperature=0.0),
            dict(top_k=1000, temperature=1.5), dict(top_p=0.0), dict(top_k=100000000, top_p=2.0, min_p=-1.0),
            dict(temperature=0.05), dict(temperature=30.0, top_p=0.3), dict(top_k=3, top_p=0.999999)]


@pytest.mark.parametrize("v,stride", [(1, 1), (2, 2), (5, 9), (31, 31), (64, 64), (1000, 1001), (4096, 4096), (4097, 4104),
                                      (8200, 8200), (16391, 16391), (50001, 50001), (151936, 151936)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_against_the_definition(v, stride, dtype):
    """Every setting on one row each, strides that leave rows unaligned, values behind the vocabulary that win if read."""
    l, u = rows(len(SETTINGS), v, v + stride, dtype, stride=stride)
    l[:, v:] = 1e4
    full = dict(temperature=1.0, top_k=0, top_p=1.0, min_p=0.0)
    compare(l, u, vocab=v, **{n: [{**full, **s}[n] for s in SETTINGS] for n in full})


def test_largest_vocabulary():
    for dtype in (torch.bfloat16, torch.float32):
        l, u = rows(3, 262144, 5, dtype, spread=0.5)
        compare(l, u, temperature=[1.0, 1.0, 0.9], top_p=[1.0, 0.97, 0.7], top_k=[0, 0, 30000])


@pytest.mark.parametrize("spread", [0.0, 1e-6, 0.01, 1.0, 20.0])
def test_many_rows_of_the_whole_distribution(spread):
    """The border between two tokens has to be where the definition has it: near flat rows have thousands of borders."""
    l, u = rows(300, 5000, 17, spread=spread)
    compare(l, u)
    l, u = rows(100, 5000, 18, spread=spread)
    compare(l, u, top_p=[0.9] * 100, temperature=[0.9] * 100)


def test_borders_of_equal_tokens():
    """Equal logits share the line evenly: u on a border belongs to the token behind it."""
    for v in (1, 2, 8, 64, 4096, 32768):
        n = min(v, 64)
        l = torch.full((n, v), -3.0, device=DEV)
        u = [j / n for j in range(n)]
        tokens, _ = call(l, u)
        assert tokens == [j * (v // n) for j in range(n)]
        below = [max(0.0, float(np.nextafter(np.float32(x), np.float32(0)))) for x in u[1:]]
        if below:
            assert call(l[1:], below)[0] == [j * (v // n) - 1 for j in range(1, n)]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_equal_logits_go_by_index(dtype):
    """Cuts inside a run of equal logits keep its first ones, wherever the run lies."""
    v = 20000
    g = torch.Generator(device=DEV).manual_seed(2)
    l = torch.full((24, v), -4.0, device=DEV)
    at = torch.randperm(v, generator=g, device=DEV)[:6000]
    l[:, at] = 1.0
    l[:, at[:20]] = 2.0
    u = torch.rand(24, generator=g, device=DEV).tolist()
    u[:3] = [0.0, 0.5, 1 - 2.0 ** -24]
    top_k = [1, 19, 20, 21, 22, 23, 500, 1777, 3000, 6019, 6020, 6021] * 2
    compare(l.to(dtype), u, top_k=top_k)
    compare(l.to(dtype), u, top_k=top_k, top_p=[0.3, 0.55, 0.8, 0.91, 0.99, 0.999] * 4)


def test_zeros_of_both_signs_are_equal():
    l = torch.tensor([[0.0, -0.0, 0.0, -0.0]] * 4, device=DEV)
    compare(l, [0.1, 0.4, 0.6, 0.9])
    assert call(l, [0.9] * 4, top_k=[1, 2, 3, 4])[0] == [0, 1, 2, 3]
    assert call(-l, [0.5] * 4, temperature=[0.0] * 4)[0] == [0] * 4


def test_masked_rows():
    """-inf and the type's lowest value, rows with one token left and with none, NaN."""
    v, inf = 9000, float("inf")
    l, u = rows(10, v, 3)
    l[0, :] = -inf
    l[1, :] = -inf
    l[1, 8765] = -80.0
    l[2, : v // 2] = -inf
    l[3, 1::2] = torch.finfo(torch.float32).min
    l[4, :] = torch.finfo(torch.float32).min
    l[5, ::3] = float("nan")
    l[6, :] = float("nan")
    l[7, 5:] = -inf
    l[8, 100:] = -3.0e38
    l[8, :100] = 3.0e38
    l[9, 0] = -inf
    for s in ({}, dict(top_k=[3] * 10), dict(top_p=[0.6] * 10), dict(temperature=[0.0] * 10),
              dict(top_k=[100] * 10, top_p=[0.9] * 10, min_p=[0.1] * 10, temperature=[0.6] * 10)):
        compare(l, u, **s)
    b = l.to(torch.bfloat16)
    b[3, 1::2] = torch.finfo(torch.bfloat16).min
    b[4, :] = torch.finfo(torch.bfloat16).min
    compare(b, u)


def test_infinite_logits_win():
    l, u = rows(2, 700, 4)
    l[:, 300], l[:, 20] = float("inf"), float("inf")
    assert call(l, u, logprobs=False)[0] == [20, 20]


def test_random_numbers_at_their_ends():
    l, _ = rows(6, 3000, 9)
    last = 1 - 2.0 ** -24
    compare(l, [0.0, last, 0.0, last, 0.0, last], top_k=[0, 0, 7, 7, 1, 1])
    # 1 and more count as the largest below 1; the row still gives a token
    tokens, _ = call(l, [1.0, 2.0, float("inf"), -1.0, float("nan"), 0.5])
    want, _ = call(l, [last, last, last, 0.0, 0.0, 0.5])
    assert tokens == want


def test_settings_at_their_ends():
    l, u = rows(6, 3000, 10)
    l = l.to(torch.bfloat16)
    top = l.float().argmax(-1).tolist()
    assert call(l, u, temperature=[1e-38, 2.0 ** -101, -1.0, float("nan"), 0.0, 1e-31])[0] == top
    compare(l, u, temperature=[2.0 ** -99] * 6)
    assert call(l, u, min_p=[1.5] * 6)[0] == call(l, u, min_p=[1.0] * 6)[0]
    assert call(l, u, top_p=[-1.0] * 6)[0] == call(l, u, top_k=[1] * 6)[0]
    compare(l, u, temperature=[1e30] * 6)


@pytest.mark.parametrize("d", [1e-3, 0.1, 1.0, 5.0, 12.0])
def test_weights_are_the_exponentials(d):
    """Two tokens: the border is at 1 / (1 + exp(-d)), asked on both sides of it at fp32's spacing."""
    border = 1 / (1 + np.exp(-float(np.float32(d))))
    u = [np.float32(border)]
    for _ in range(4):
        u.append(np.nextafter(u[-1], np.float32(1)))
    for _ in range(4):
        u.append(np.nextafter(u[0] if len(u) == 5 else u[-1], np.float32(0)))
    l = torch.tensor([[d, 0.0]] * 9, device=DEV)
    tokens, _ = call(l, [float(x) for x in u])
    assert tokens == [int(float(x) >= border) for x in u]


def test_captured_calls_and_several_streams():
    b, v = 40, 30001
    l, u = rows(b, v, 6)
    u = torch.tensor(u, device=DEV)
    p, t = torch.full((b,), 0.9, device=DEV), torch.full((b,), 0.8, device=DEV)
    want = nf4.sample(l, u, t, None, p)
    tokens = torch.zeros(b, dtype=torch.int32, device=DEV)
    logs = torch.zeros(b, device=DEV)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        nf4.nf4_sample(l, u, tokens, t, None, p, logprobs=logs)
    for _ in range(3):
        tokens.zero_()
        graph.replay()
        assert torch.equal(tokens, want[0]) and torch.equal(logs, want[1])
    # inputs change between replays
    u2 = torch.rand(b, device=DEV)
    u.copy_(u2)
    graph.replay()
    again = nf4.sample(l, u2, t, None, p)
    assert torch.equal(tokens, again[0])
    streams = [torch.cuda.Stream() for _ in range(4)]
    torch.cuda.synchronize()
    got = [nf4.sample(l, u, t, None, p, stream=s) for s in streams for _ in range(3)]
    torch.cuda.synchronize()
    for g in got:
        assert torch.equal(g[0], again[0]) and torch.equal(g[1], again[1])


@pytest.mark.parametrize("v", [9, 700, 30011])
@pytest.mark.parametrize("settings", [{}, dict(top_k=[5] * 3), dict(temperature=[0.0] * 3), dict(top_p=[0.5] * 3)])
def test_infinite_logits_have_equal_shares(v, settings):
    """log softmax of a row with n infinite logits is -log n at each; one row's infinities are in two slices."""
    l, u = rows(3, v, 4)
    l[0, v // 2] = l[1, v - 1] = l[1, 2] = l[2, 0] = float("inf")
    l[2, 1::2] = -float("inf")
    tokens, logs = call(l, u, **settings)
    assert tokens == [v // 2, 2, 0]
    assert logs[0] == 0.0 and abs(logs[1] + np.log(2.0)) <= 2.0 ** -24 and logs[2] == 0.0
