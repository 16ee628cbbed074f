"""The attention at the limits of what it accepts (GPU)."""
import pytest
import torch

from test_layer_ops_gpu import FORMATS, check, new_cache, randn

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("group", [2, 12])
def test_longest_lengths(fmt, group):
    """max_pages * page_size = 2^31 - 16, the most that is accepted, and lengths up to it; a window leaves the last
    keys, so that only the last two pages of each sequence need be there."""
    page, max_pages = 8176, 262657
    assert page * max_pages == 2 ** 31 - 16
    lengths = [2 ** 31 - 16, 2 ** 31 - 17, 2 ** 31 - 40, 2 ** 31 - 8191]
    c = new_cache(fmt, 3, 1, page, 64, seed=5)
    table = torch.full((len(lengths), max_pages), -1, dtype=torch.int32)
    table[:, -2:] = torch.tensor([[2, 0], [1, 2], [0, 1], [1, 0]], dtype=torch.int32)
    check(c, randn((len(lengths), group, 64), 6), table, lengths, window=300)
    check(c, randn((len(lengths), group, 64), 7), table, lengths, window=33)
