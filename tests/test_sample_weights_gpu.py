"""The weights that nf4_sample draws by (GPU): 2^40 exp((l - max l) / T) as a whole number, within 1.1 * 2^-30 of its
size or half a multiple.

The bound, in units of 2^-30 of a weight: the table's entry is off by half a unit (it has 31 bits, and is 2^30 or more), the
rounded correction by another half; the correction is below 2^-11.5 of the weight and passes four roundings of fp32, 2^-24 of
it each (0.1 in all), a term of 2^-37 that its series leaves out and a product cut at 1/256 of a unit."""
from fractions import Fraction

import numpy as np
import pytest
import torch

import nf4_weight_only_gb300 as nf4

from gpu_util import DEV

pytestmark = pytest.mark.gpu

UNIT = 2.0 ** -30


def tokens_of(logits, u, **settings):
    b = logits.shape[0]
    tokens = torch.zeros(b, dtype=torch.int32, device=DEV)
    nf4.nf4_sample(logits, torch.tensor(u, dtype=torch.float32, device=DEV), tokens, **settings)
    return tokens.cpu().numpy()


@pytest.mark.parametrize("heat", [1.0, 0.7, 1.7])
@pytest.mark.parametrize("short", [False, True])
def test_borders_between_two_tokens(heat, short):
    """Two tokens, the first with the weight w = exp(-d / T): the border is at w / (1 + w), so a weight that is off by e of
    itself moves it by e / (1 + w) of itself.  Asked are random numbers that lie 1.1 to 1.6 units from the border, of which
    every hundredth pair of fp32 numbers gives one.  Weights above 2^-10 are multiples of 2^-40 without a further rounding."""
    rng = np.random.default_rng(11)
    t = float(np.float32(heat))
    d = rng.uniform(1e-4, 6.0 * t, 1 << 21).astype(np.float32)
    w = np.exp(-d.astype(np.float64) / t)
    border = w / (1 + w)
    u = border.astype(np.float32)
    off = (u.astype(np.float64) - border) / border * (1 + w) / UNIT
    ask = (np.abs(off) > 1.1) & (np.abs(off) < 1.6)
    assert ask.sum() > 4000 and w.min() > 2.0 ** -10
    d, u, off = d[ask], u[ask], off[ask]
    # (the short way needs a top_k below the number of tokens)
    width = 3 if short else 2
    l = torch.full((len(d), width), -float("inf"), device=DEV)
    l[:, 0], l[:, 1] = -torch.from_numpy(d).to(DEV), 0.0
    more = dict(top_k=torch.full((len(d),), 2, dtype=torch.int32, device=DEV)) if short else {}
    got = tokens_of(l, u, temperature=torch.full((len(d),), t, device=DEV), **more)
    wrong = np.nonzero(got != (off > 0))[0]
    assert len(wrong) == 0, (len(wrong), len(d), off[wrong[:5]])


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("tail", [-28.5, -28.0, -27.0, -26.0, -25.0])
def test_long_tails(dtype, tail):
    """One likely token and 262143 equal ones far below, whose weights are a few multiples of 2^-40, or none: below half a
    multiple they are never drawn, else every one of them as often as its multiples say."""
    v, top = 262144, 70001
    each = int(np.floor(np.exp(tail) * 2.0 ** 40 + 0.5))
    assert abs(np.exp(tail) * 2.0 ** 40 % 1 - 0.5) > 0.01 and (each == 0) == (tail == -28.5)
    u = np.array([0.0, 2.0 ** -20, 0.3, 0.5, 1 - 2.0 ** -10, 1 - 2.0 ** -23, 1 - 2.0 ** -24], np.float32)
    l = torch.full((len(u), v), tail, device=DEV)
    l[:, top] = 0.0
    got = tokens_of(l.to(dtype), u)
    total = 2 ** 40 + (v - 1) * each
    for x, token in zip(u, got):
        goal = int(Fraction(float(x)) * total)  # the first token whose sum passes it
        before = top * each
        if goal < before:
            want = goal // each
        elif goal < before + 2 ** 40:
            want = top
        else:
            want = top + 1 + (goal - before - 2 ** 40) // each
        assert token == want, (float(x), token, want)
