"""The attention at the limits of what it accepts (GPU)."""
import pytest
import torch

import nf4_weight_only_gb300 as nf4
from gpu_util import DEV
from test_layer_ops_gpu import FORMATS, check, new_cache, paged, randn

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


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("batch", [7, 45])
def test_a_batch_cut_anywhere(fmt, batch):
    """The rows of a batch from any of them on: the same bytes, wherever lengths, page table and positions begin."""
    g = torch.Generator().manual_seed(batch)
    lengths = torch.randint(0, 300, (batch,), generator=g).tolist()
    page, wide = 16, 19
    need = sum(-(-n // page) for n in lengths)
    c = new_cache(fmt, need, 2, page, 64, seed=5)
    table = paged(lengths, page, need, wide, 6).to(DEV)
    q, n = randn((batch, 4, 64), 7), torch.tensor(lengths, dtype=torch.int32, device=DEV)
    positions, freq = (n * 37)[None], torch.rand(32, device=DEV)
    ws = nf4.attention_workspace(c, batch, 4)
    whole = nf4.attention_decode(c, q, table, n, ws)
    turned, _ = nf4.rope(q, q[:, :2].contiguous(), positions, freq)
    for i in range(1, 6):
        assert torch.equal(nf4.attention_decode(c, q[i:], table[i:], n[i:], ws), whole[i:])
        assert torch.equal(nf4.rope(q[i:], q[i:, :2].contiguous(), positions[:, i:], freq)[0], turned[i:])
    assert nf4.nf4_check_device_error() == 0
