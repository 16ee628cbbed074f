"""The residual norm and the rotary positions where their forms and ranges end (GPU)."""
import pytest
import torch

import nf4_weight_only_gb300 as nf4
from gpu_util import DEV, Guarded
from test_layer_ops_gpu import randn

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("rows,width", [(4, 64), (700, 2056), (700, 5120)])
@pytest.mark.parametrize("eps", [1e-6, 1.0])
@pytest.mark.parametrize("top", [1e-35, 1e-36, 4e-37, 1e-38, 1e-39, 2e-40, 1e-40])
def test_norm_scale_below_its_reciprocals_range(rows, width, top, eps):
    """Rows whose largest value makes a scale at or below 2^-126, beside zeros: codes of y / s, and no NaN.

    s = fp32(max |y| / 448) is off by up to 2^-150 where it is subnormal; y / s has that relative error too, and a code
    is within half a step of it.  (With eps = 1e-6 the smallest tops are of inputs that round to 0: s = 0.)"""
    x = torch.zeros((rows, width), device=DEV)
    # 448 / s at 0, then values of every size down to it, zeros between
    n = torch.arange(width, device=DEV)
    x[:] = torch.where(n % 3 == 0, 0.0, 1.0 / (1 + n % 61)) * torch.where(n % 2 == 0, 1.0, -1.0)
    x[:, 1] = 1
    # y = x rsqrt(eps): eps is all of the mean square
    x = (x * (top * eps ** 0.5)).to(torch.bfloat16)
    w = torch.ones(width, dtype=torch.bfloat16, device=DEV)
    y8, s = Guarded((rows, width), torch.float8_e4m3fn), Guarded((rows,), torch.float32)
    nf4.nf4_rmsnorm(x, w, eps, y8=y8.t, y8_scales=s.t)
    assert y8.canaries_intact() and s.canaries_intact()
    want = x.double() * (1 / torch.tensor(eps, dtype=torch.float32).double().sqrt().item())
    s64 = want.abs().amax(-1) / 448
    assert bool(((s.t.double() - s64).abs() <= 2.0 ** -20 * s64 + 2.0 ** -149).all())
    codes = y8.t.float().double()
    assert not codes.isnan().any() and not codes[x == 0].any()
    # y itself is fp32: a subnormal one is off by up to 2^-150
    ratio = torch.where(s.t[:, None] > 0, want / s.t.double()[:, None], 0.0)
    slack = 2.0 ** -18 * ratio.abs() + 2.0 ** -149 / s.t.double()[:, None]
    step = torch.maximum(2.0 ** -4 * ratio.abs(), torch.full_like(ratio, 2.0 ** -10))
    assert bool(((codes - ratio.clamp(-448, 448)).abs() <= step + slack).all())


@pytest.mark.parametrize("rows,width", [(4, 64), (700, 2056), (2, 40000)])
def test_norm_of_zero_rows_without_eps(rows, width):
    """An all-zero row gives zeros, scale 0 and codes 0 for any eps, 0 too."""
    x, w = randn((rows, width), 1), randn((width,), 2)
    x[1] = 0
    y, y8 = Guarded(x.shape, torch.bfloat16), Guarded(x.shape, torch.float8_e4m3fn)
    s = Guarded((rows,), torch.float32)
    nf4.nf4_rmsnorm(x, w, 0.0, y=y.t, y8=y8.t, y8_scales=s.t)
    assert y.canaries_intact() and y8.canaries_intact() and s.canaries_intact()
    assert not y.t[1].any() and not y8.t[1].float().any() and float(s.t[1]) == 0.0
    h = x.double()
    want = h / (h * h).mean(-1, keepdim=True).sqrt().clamp_min(1e-300) * w.double()
    assert bool(((y.t.double() - want).abs() <= 2.0 ** -8 * want.abs()).all())
