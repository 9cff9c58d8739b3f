"""Group norm of values beyond 16, where the exact sums take the wide steps: the statistics do not depend on the patches or
on the frame's kernels, and a value out of range is flagged wherever it lies among the 32 that a thread sums together."""
import numpy as np
import pytest
import torch

from oracle import plan

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def vd():
    from patch_tiled_causal_gb300 import build, vaedec
    build.build()
    vaedec.load()
    vaedec.last_error()
    return vaedec


def norm(vd, x, groups, nph, npw):
    B, T, H, W, Cc = x.shape
    d = vd.gn_desc(B, T, H, W, Cc, groups, plan.band_edges(H, nph), plan.band_edges(W, npw), silu=False,
                   in_dtype=vd.VAE_FP32 if x.dtype == torch.float32 else vd.VAE_BF16, out_dtype=vd.VAE_FP32)
    y = torch.full(x.shape, float("nan"), device="cuda")
    ws = vd.gn_workspace(d, "cuda")
    vd.patch_groupnorm_silu(x, torch.ones(Cc, device="cuda"), torch.zeros(Cc, device="cuda"), y, ws, d)
    return y


@pytest.mark.parametrize("dt", ["bf16", "fp32"])
@pytest.mark.parametrize("shape,groups", [((1, 2, 24, 40, 256), 32), ((1, 2, 19, 23, 64), 32), ((2, 1, 17, 31, 32), 32), ((1, 1, 9, 30, 128), 64),
                                          ((1, 1, 5, 40, 1024), 32)])
@pytest.mark.parametrize("top", [15.9, 17.0, 8191.0])
def test_large_values_do_not_depend_on_the_patches(vd, dt, shape, groups, top):
    gen = torch.Generator(device="cuda").manual_seed(1)
    x = (torch.randn(shape, generator=gen, device="cuda") * top / 3).clamp(-top, top).to(torch.bfloat16 if dt == "bf16" else torch.float32)
    x = x.clamp(-8160, 8160)  # (the bf16 number below 8192)
    want = norm(vd, x, groups, 1, 1)
    for nph, npw in ((2, 2), (4, 5), (1, 20), (shape[2], 1)):
        assert torch.equal(norm(vd, x, groups, nph, npw), want), (nph, npw)
    assert vd.last_error()[0] == vd.VAE_OK
    # the formula in 64 bits; x enters the sums in steps of 2^-18, and y = a x + s rounds a, mean a, s and the result
    g = x.double().reshape(*shape[:4], groups, -1)
    var, mean = torch.var_mean(g, dim=(2, 3, 5), correction=0, keepdim=True)
    a = 1 / torch.sqrt(var + 1e-6)
    ref = ((g - mean) * a).reshape(shape)
    tol = (6 * 2.0 ** -24 * ((g * a).abs() + (mean * a).abs()) + 2.0 ** -19 * a * (1 + (g - mean).abs() * a)).reshape(shape)
    assert ((want.double() - ref).abs() <= tol).all()


@pytest.mark.parametrize("bad", [8192.0, -8200.0, float("nan"), float("inf")])
def test_a_value_out_of_range_is_flagged_wherever_it_lies(vd, bad):
    x = torch.ones((1, 1, 5, 40, 64), device="cuda")
    for h, w, c in ((0, 0, 0), (0, 9, 7), (2, 31, 8), (4, 39, 63), (4, 0, 33)):
        y = x.clone()
        y[0, 0, h, w, c] = bad
        norm(vd, y, 8, 2, 3)
        assert vd.last_error()[0] == vd.VAE_ERR_RANGE, (h, w, c)
        norm(vd, x, 8, 2, 3)
        assert vd.last_error()[0] == vd.VAE_OK
