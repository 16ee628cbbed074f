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


def two_pi_inverse():
    """floor(2^400 / (2 pi)), by Machin's formula for pi."""
    bits = 700

    def arctan_inverse(n):  # 2^bits * arctan(1 / n)
        total, power, k = 0, (1 << bits) // n, 0
        while power:
            total += (-1) ** k * (power // (2 * k + 1))
            power //= n * n
            k += 1
        return total

    pi = 4 * (4 * arctan_inverse(5) - arctan_inverse(239))
    return (1 << (400 + bits)) // (2 * pi)


def turn(position, frequency):
    """position * frequency radians as a fraction of a turn in [0, 1), in integers."""
    n, d = float(frequency).as_integer_ratio()  # d: a power of two
    return (position * n * two_pi_inverse() // d) % (1 << 400) / (1 << 400)


FREQUENCIES = [255.0, 255.99998, 256.0, 257.5, 511.0, 1000.0, 65535.0, 1e6, 3.3e7, 1e10, 1e19, 1e25, 1e30, 2.0 ** 104, 1e38,
               2.0 ** 127, 3.4028234e38, -256.0, -1e6, -3.4e38, 1.0, 0.0, 1e-30, 1e-45, -0.75, 2.0 ** 24 - 1, 16777215.0 * 64,
               300.25, 1e3 / 3, 2e4, 7e8, 5e14]


@pytest.mark.parametrize("inter", [False, True])
def test_rope_of_large_frequencies(inter):
    """The angle is the real product at any frequency and position: against integers of 400 bits."""
    assert len(FREQUENCIES) == 32
    positions = [0, 1, -1, 2, 3, 1000, 131071, 2 ** 31 - 1, -(2 ** 31), -98765]
    inv = torch.tensor(FREQUENCIES, dtype=torch.float32)
    angle = torch.tensor([[turn(p, f) for f in inv.tolist()] for p in positions], dtype=torch.float64, device=DEV)
    cos, sin = (angle * 2 * torch.pi).cos()[:, None], (angle * 2 * torch.pi).sin()[:, None]
    q, k = randn((len(positions), 3, 64), 1), randn((len(positions), 1, 64), 2)
    at = torch.tensor([positions], dtype=torch.int32, device=DEV)
    for x, got in zip((q, k), nf4.rope(q, k, at, inv.to(DEV), interleaved=inter)):
        x, got = x.double(), got.double()
        first, second = (slice(0, 64, 2), slice(1, 64, 2)) if inter else (slice(0, 32), slice(32, 64))
        a, b = x[..., first], x[..., second]
        slack = 2.0 ** -18 * (a.abs() + b.abs())
        for want, part in ((a * cos - b * sin, first), (b * cos + a * sin, second)):
            assert bool(((got[..., part] - want).abs() <= 2.0 ** -8 * want.abs() + slack).all())


SMS = torch.cuda.get_device_properties(0).multi_processor_count if torch.cuda.is_available() else 152


@pytest.mark.parametrize("rows", [4 * SMS, 4 * SMS + 1, 9 * SMS + 5, 13 * SMS - 3])
@pytest.mark.parametrize("width", [2048, 2056, 3080, 5120, 5128, 8184, 8192, 8200])
@pytest.mark.parametrize("residual", [True, False])
def test_norm_of_many_rows(rows, width, residual):
    """Rows that go through persistent CTAs (more than 4 an SM, more than 2048 and up to 8192 wide), several a CTA with
    an uneven last turn, and the neighbours of these limits: every output alone, all of them, and in place."""
    x, w = randn((rows, width), 1), (1 + 0.2 * randn((width,), 2).float()).to(torch.bfloat16)
    r = randn((rows, width), 3, 4.0) if residual else None
    size = torch.exp2(((torch.arange(rows, device=DEV) * 7) % 19 - 9).float())[:, None]  # no two rows in turn alike
    x = (x.float() * size).to(torch.bfloat16)
    x[5] = 0
    if residual:
        r = (r.float() * size).to(torch.bfloat16)
        r[5] = 0
    h32 = x.float() + r.float() if residual else x.float()
    h, eps = h32.double(), 1e-6
    want = h / torch.sqrt((h * h).mean(-1, keepdim=True) + eps) * w.double()
    s64 = want.abs().amax(-1) / 448
    ro, y = Guarded(x.shape, torch.bfloat16), Guarded(x.shape, torch.bfloat16)
    y8, sc = Guarded(x.shape, torch.float8_e4m3fn), Guarded((rows,), torch.float32)
    nf4.nf4_rmsnorm(x, w, eps, residual=r, residual_out=ro.t, y=y.t, y8=y8.t, y8_scales=sc.t)
    assert all(g.canaries_intact() for g in (ro, y, y8, sc))
    assert torch.equal(ro.t, h32.to(torch.bfloat16))
    # bf16's rounding, and 2^-20 for the fp32 sum, root and products
    assert bool(((y.t.double() - want).abs() <= (2.0 ** -8 + 2.0 ** -20) * want.abs()).all())
    assert bool(((sc.t.double() - s64).abs() <= 2.0 ** -20 * s64).all())
    step = torch.maximum(2.0 ** -4 * want.abs(), 2.0 ** -10 * s64[:, None])
    assert bool(((y8.t.float().double() * sc.t.double()[:, None] - want).abs() <= step * (1 + 2.0 ** -10)).all())
    # alone, and in place: the same bytes
    one, one8, ones = torch.empty_like(x), torch.empty_like(y8.t), torch.empty_like(sc.t)
    nf4.nf4_rmsnorm(x, w, eps, residual=r, y=one)
    assert torch.equal(one, y.t)
    nf4.nf4_rmsnorm(x, w, eps, residual=r, y8=one8, y8_scales=ones)
    assert torch.equal(one8.view(torch.uint8), y8.t.view(torch.uint8)) and torch.equal(ones, sc.t)
    a, b = x.clone(), None if r is None else r.clone()
    nf4.nf4_rmsnorm(a, w, eps, residual=b, residual_out=b, y=a)
    assert torch.equal(a, y.t) and (b is None or torch.equal(b, ro.t))
    a = x.clone()
    nf4.nf4_rmsnorm(a, w, eps, residual=r, residual_out=a, y8=one8, y8_scales=ones)
    assert torch.equal(a, ro.t) and torch.equal(one8.view(torch.uint8), y8.t.view(torch.uint8))
