"""The log-probabilities of nf4_sample where their sum is hardest (GPU): within 2^-17 + 2^-22 of their size.

With S = n + rest, n the number of largest logits, counted, and rest the sum of the others' exp(-x): log S is off by
rest / S times the relative error of rest.  That is at most 80 additions of fp32 one after the other (40 of a thread's pairs in the largest
slice, 40 over threads, warps and slices), 2^-24 of the sum each; and of a term the error of x log2(e) in fp32,
2^-24 x / ln 2 twice, and of the hardware's exp2, 2^-22.  rest / S is at most half for x of 12.5 and more (262144 tokens), so
80 * 2^-24 + 12.5 * 2^-24 * 2 + 2^-22 < 2^-17 in all; the subtraction of log S rounds by 2^-24 of the result."""
import numpy as np
import pytest
import torch

import nf4_weight_only_gb300 as nf4

from gpu_util import DEV

pytestmark = pytest.mark.gpu


def compare(logits, u):
    b = logits.shape[0]
    tokens, logs = torch.zeros(b, dtype=torch.int32, device=DEV), torch.zeros(b, device=DEV)
    nf4.nf4_sample(logits, u, tokens, logprobs=logs)
    want = torch.log_softmax(logits.double(), -1).gather(1, tokens.long()[:, None])[:, 0]
    bound = 2.0 ** -17 + 2.0 ** -22 * want.abs()
    assert bool(((logs.double() - want).abs() <= bound).all()), float((logs.double() - want).abs().max())
    return tokens


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("v,b", [(262144, 1), (262144, 40), (151936, 1), (151936, 200), (40960, 300), (3001, 5)])
@pytest.mark.parametrize("x", [0.5, 3.0, 8.1, 11.3, 12.5, 20.0])
def test_many_equal_tails(dtype, v, b, x):
    """Equal terms round alike in every addition."""
    l = torch.full((b, v), -x, device=DEV).to(dtype)
    l[:, v // 3] = 0.0
    u = torch.rand(b, generator=torch.Generator(device=DEV).manual_seed(v + b), device=DEV)
    u[0] = 0.9999
    compare(l, u)


@pytest.mark.parametrize("gap", [12.0, 14.0, 16.0, 20.0, 30.0])
def test_probabilities_near_one(gap):
    """-log(1 + e), e of 6e-6 to 1e-13: the counted top keeps its digits, so the error is a share of e."""
    for n in (1, 7, 1000):
        l = torch.full((3, 5000), -200.0, device=DEV)
        l[:, 100:100 + n] = -gap
        l[:, 4000] = 0.0
        tokens, logs = torch.zeros(3, dtype=torch.int32, device=DEV), torch.zeros(3, device=DEV)
        nf4.nf4_sample(l, torch.full((3,), 0.5, device=DEV), tokens, logprobs=logs)
        e = n * np.exp(-gap)
        assert tokens.tolist() == [4000] * 3
        # (1000 terms: 80 additions at most; x log2(e) and exp2 as above; the logarithm's own rounding)
        share = 80 * 2.0 ** -24 + gap * 2.0 ** -23 + 2.0 ** -22 + 2.0 ** -22
        assert all(abs(x + np.log1p(e)) <= share * e for x in logs.double().tolist()), (logs.tolist(), -np.log1p(e))
