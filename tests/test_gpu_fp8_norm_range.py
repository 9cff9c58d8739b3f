"""The RMS norm of a residual sum where a row's squares lie near or below fp32's smallest numbers, through the C ABI.

Rows of values +-m come out as +-m / sqrt(m^2 + eps), whose blocks have that over 448 as their scale.  Off by a few fp32 units:
the mean (a sum of equal squares: each addition half a unit, up to 40 in a chain of lanes, vectors and warps, halved by the root:
20), the root, the reciprocal, two products and the scale half a unit each: 23 units of 2^-24, under 2^-19 of the value."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def vd():
    from patch_tiled_causal_gb300 import build, vaedec
    build.build()
    vaedec.load()
    vaedec.last_error()
    return vaedec


ROWS = [2.0 ** 57, 1e10, 1.0, 1e-10, 3e-16, 1e-18, 1.1e-19, 1e-19, 3e-20, 1e-20, 3e-21, 1e-22, 1e-23, 1e-30, 1e-38, 1e-40, 2.0 ** -149]


# a row per 8, 16 and 32 lanes, per thread block with two and four vectors a lane, rows off 16 bytes per warp and per thread block
@pytest.mark.parametrize("cols", [72, 200, 400, 1000, 4096, 16384, 301, 1001, 3001, 17001])
@pytest.mark.parametrize("eps", [0.0, 2.0 ** -149, 1e-40, 1e-37, 1e-31, 1e-12])
def test_tiny_rows(vd, cols, eps):
    m = torch.tensor(ROWS, device="cuda")
    wide = torch.zeros((len(m), cols + (-cols % 8 if cols % 2 == 0 else 2)), device="cuda")
    x = wide[:, :cols]
    x.copy_(m[:, None] * torch.where(torch.arange(cols, device="cuda") % 3 == 1, -1.0, 1.0))
    codes, scales = vd.fp8_empty(len(m), cols)
    total = torch.empty((len(m), cols), device="cuda")
    vd.residual_rmsnorm_silu_fp8(x, None, torch.ones(cols, device="cuda"), None, total, codes, scales, eps=eps)
    over = cols * 2.0 ** 114 >= 2.0 ** 128  # the first row's squares leave fp32 at the top: NaN
    assert vd.last_error()[0] == (vd.VAE_ERR_RANGE if over else vd.VAE_OK)
    assert torch.equal(total, x)
    assert bool(torch.isnan(scales[:, 0]).all()) == over
    m, scales = m[1:].double(), scales[:, 1:].double()
    want = torch.clamp(m / torch.sqrt(m * m + float(np.float32(eps))) / 448.0, min=2.0 ** -126)
    assert bool(((scales - want).abs() <= 2.0 ** -19 * want).all())


@pytest.mark.parametrize("cols", [72, 400, 4096, 301, 3001])
def test_rows_of_all_sizes_beside_each_other(vd, cols):
    # rows that share a warp, one of them tiny: each as by itself
    m = torch.tensor([1.0, 1e-22, 0.0, 3.0, 1e-30, 1e-5, 1e-21] * 9, device="cuda")
    x = torch.randn((len(m), cols), device="cuda", generator=torch.Generator(device="cuda").manual_seed(1)) * m[:, None]
    g = torch.ones(cols, device="cuda")
    codes, scales = vd.fp8_empty(len(m), cols)
    vd.residual_rmsnorm_silu_fp8(x, None, g, None, None, codes, scales, eps=1e-44)
    assert vd.last_error()[0] == vd.VAE_OK
    for r in range(len(m)):
        c, s = vd.fp8_empty(1, cols)
        vd.residual_rmsnorm_silu_fp8(x[r:r + 1], None, g, None, None, c, s, eps=1e-44)
        assert torch.equal(c.view(torch.uint8)[0], codes.view(torch.uint8)[r]) and torch.equal(s[:, 0], scales[:, r])


def test_zero_rows(vd):
    x, codes, scales = torch.zeros((3, 200), device="cuda"), *vd.fp8_empty(3, 200)
    for eps in (1e-6, 1e-30, 1e-40, 2.0 ** -149):
        vd.residual_rmsnorm_silu_fp8(x, None, torch.ones(200, device="cuda"), None, None, codes, scales, eps=eps)
        assert vd.last_error()[0] == vd.VAE_OK and bool((scales == 2.0 ** -126).all())
    vd.residual_rmsnorm_silu_fp8(x, None, torch.ones(200, device="cuda"), None, None, codes, scales, eps=0.0)  # 0 / 0
    assert vd.last_error()[0] == vd.VAE_ERR_RANGE and bool(torch.isnan(scales).all())
