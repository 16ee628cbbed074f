"""nf4_lora beside a projection of as many rows as the call takes (GPU; 69 GB of B): columns up to the last are computed and
copied.  The bound on y is that of rank 16: 2^-8 of it, and 2^-16 + (16 + 64) * 2^-23 of the sum of the terms' sizes (one k of
x counts, so h is exact)."""
import pytest
import torch

import nf4_weight_only_gb300 as nf4

from gpu_util import DEV

pytestmark = pytest.mark.gpu

EDGE = 4096  # columns at both ends in which B is not zero


@pytest.mark.parametrize("n", [(1 << 31) - 8, (1 << 31) - 1])
def test_columns_up_to_the_last(n):
    """A token with an adapter and one without; rows of 16-byte pieces and rows that begin anywhere."""
    torch.cuda.empty_cache()
    if torch.cuda.mem_get_info()[0] < 110 << 30:
        pytest.skip("needs 110 GB of device memory")
    bf = torch.bfloat16
    g = torch.Generator(device=DEV).manual_seed(n % 1000)
    b = torch.zeros((1, n, 16), dtype=bf, device=DEV)
    for at in (0, n - EDGE):
        b[0, at:at + EDGE] = torch.randn((EDGE, 16), generator=g, device=DEV).to(bf)
    base = torch.empty((2, n), dtype=bf, device=DEV).normal_(generator=g)
    y = torch.full((2, n), 77.0, dtype=bf, device=DEV)
    x = torch.zeros((2, 64), dtype=bf, device=DEV)
    x[0, 5] = 1.0
    a = torch.randn((1, 16, 64), generator=g, device=DEV).to(bf)
    scales = torch.tensor([0.5], device=DEV)
    plan = nf4.lora_plan(torch.tensor([0, -1], dtype=torch.int32, device=DEV), 1)
    nf4.nf4_lora(x, plan, scales, [a], [b], [y], nf4.lora_workspace(2, 1, 16, 1), bases=[base])
    assert nf4.nf4_check_device_error() == 0
    # (a sum of exact comparisons; torch.equal would hold both rows once more)
    step = 1 << 28
    assert all(torch.equal(y[1, i:i + step], base[1, i:i + step]) for i in range(0, n, step))
    assert all(torch.equal(y[0, i:i + step], base[0, i:i + step])
               for i0 in range(EDGE, n - EDGE, step) for i in [i0] if i + step <= n - EDGE)
    h = 0.5 * a[0, :, 5].double()
    for at in (0, n - EDGE):
        rows = b[0, at:at + EDGE].double()
        want = base[0, at:at + EDGE].double() + rows @ h
        bound = 2.0 ** -8 * want.abs() + (rows.abs() @ h.abs()) * (2.0 ** -16 + 80 * 2.0 ** -23) + \
            2.0 ** -22 * base[0, at:at + EDGE].double().abs()
        assert bool(((y[0, at:at + EDGE].double() - want).abs() <= bound).all())
    del b, base, y
    torch.cuda.empty_cache()
