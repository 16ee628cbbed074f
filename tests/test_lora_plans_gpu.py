"""Plans for nf4_lora whose words were overwritten (GPU): a chunk outside the lists is left out, the others are computed."""
import pytest
import torch

import nf4_weight_only_gb300 as nf4

from gpu_util import DEV
from test_lora_gpu import Case

pytestmark = pytest.mark.gpu

MOST = (1 << 31) - 1


@pytest.mark.parametrize("many", [True, False])
@pytest.mark.parametrize("words", [(0, MOST, 1), (0, MOST - 15, 16), (0, MOST - 63, 64), (0, -1, 4), (0, 0, MOST), (0, 0, -MOST),
                                   (3, 0, 4), (MOST, 0, 4), (-1, 0, 4)])
def test_chunks_outside_the_lists_are_left_out(many, words):
    # adapter 0 has one chunk, adapter 1 another of the same kind
    n = 40 if many else 9
    c = Case(2 * n, 192, [72, 40], 16, 3, [0] * n + [1] * n, seed=n)
    plan = c.plan.view(torch.int32)
    assert plan[2:4].tolist() == ([2, 0] if many else [0, 2]) and plan[8:11].tolist() == [0, 0, n]
    plan[8:11] = torch.tensor(words, dtype=torch.int32)
    for y in c.ys:
        y.t.fill_(3.0)
    c.run()
    for y in c.ys:
        assert bool((y.t[:n] == 3.0).all()) and y.canaries_intact()
    c.check(sample=range(n, 2 * n))
