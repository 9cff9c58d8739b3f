"""The RMS norm of a residual sum over so many rows that blocks go over them with gamma and beta in shared memory (more
groups of rows than 16 times the SMs), through the C ABI.

Each row's result is the one that a call of few rows gives, bit for bit (the same arithmetic in the same order, with the
parameters read from elsewhere), and some rows are compared with float64: with t = 1e-5 (|y| + |beta|) every value lies between
the quantised y - t and y + t at the scale that was written (the mean of squares is off by under 70 roundings of 2^-24, so its root
by 35, the rest by a few, SiLU by a few 2^-22 and |z| 2^-24 with |z| below 90: under 1e-5 in all)."""
import numpy as np
import pytest
import torch

from oracle import fp8

pytestmark = pytest.mark.gpu

T = {"bf16": torch.bfloat16, "fp32": torch.float32}
# rows and columns for rows held by 8, 16, 32 lanes and by 32 lanes with two vectors each; columns that end inside a vector
# and inside a block, and full ones; last groups of rows that are not full
SIZES = [(80001, 72), (78850, 128), (40003, 200), (39000, 256), (20011, 400), (20011, 1000), (19600, 1024)]


@pytest.fixture(scope="module")
def vd():
    from patch_tiled_causal_gb300 import build, vaedec
    build.build()
    vaedec.load()
    vaedec.last_error()
    return vaedec


def strided(x, pad):
    """x in a matrix whose rows are `pad` longer, the rest 7."""
    wide = torch.full((x.shape[0], x.shape[1] + pad), 7.0, device="cuda", dtype=x.dtype)
    wide[:, :x.shape[1]] = x
    return wide, wide[:, :x.shape[1]]


@pytest.mark.parametrize("rows,cols", SIZES)
@pytest.mark.parametrize("dt,rt", [("bf16", "bf16"), ("bf16", "fp32"), ("fp32", "bf16"), ("fp32", "fp32")])
@pytest.mark.parametrize("form", ["apart", "total is x", "total is the residual", "norm alone"])
def test_many_rows(vd, rows, cols, dt, rt, form):
    if form == "total is x" and dt != rt:
        rt = dt
    groups = -(-rows // (256 // (8 if cols <= 128 else 16 if cols <= 256 else 32)))
    assert groups > 16 * torch.cuda.get_device_properties(0).multi_processor_count
    gen = torch.Generator(device="cuda").manual_seed(rows + cols)
    size = torch.exp2(torch.linspace(-6, 6, rows, device="cuda"))[:, None]
    x = (torch.randn((rows, cols), generator=gen, device="cuda") * size).to(T[dt])
    res = (2.0 * torch.randn((rows, cols), generator=gen, device="cuda") * size).to(T[rt])
    gamma = 1.0 + 0.2 * torch.randn(cols, generator=gen, device="cuda")
    beta = 0.1 * torch.randn(cols, generator=gen, device="cuda")
    bad = rows - 300  # (a block's second row or a later one)
    x[bad, cols // 2] = float("nan")
    silu = form in ("total is x", "norm alone")
    res = None if form == "norm alone" else res
    beta = None if form in ("total is the residual", "norm alone") else beta

    def run(x, res, total):
        codes, scales = vd.fp8_empty(x.shape[0], cols)
        codes.view(torch.uint8).fill_(0xA5)
        scales.fill_(-7.0)
        vd.residual_rmsnorm_silu_fp8(x, res, gamma, beta, total, codes, scales, silu=silu)
        return codes.view(torch.uint8), scales

    (xw, xv), (rw, rv) = strided(x, 8), (None, None) if res is None else strided(res, 16)
    tw, tv = {"apart": lambda: strided(torch.zeros((rows, cols), device="cuda", dtype=T[rt]), 24), "total is x": lambda: (xw, xv),
              "total is the residual": lambda: (rw, rv), "norm alone": lambda: (None, None)}[form]()
    codes, scales = run(xv, rv, tv)
    assert vd.last_error()[0] == vd.VAE_ERR_RANGE  # (the row with the NaN)
    assert vd.last_error()[0] == vd.VAE_OK
    for w in (xw, rw, tw):
        assert w is None or bool((w[:, cols:] == 7.0).all())
    assert bool(torch.isnan(scales[:, bad]).all()) and int(torch.isnan(scales).sum()) == scales.shape[0]
    for r0 in range(0, rows, 2400):
        r1 = min(rows, r0 + 2400)
        total = None if tv is None else torch.empty((r1 - r0, cols), device="cuda", dtype=T[rt])
        c, s = run(x[r0:r1], None if res is None else res[r0:r1], total)
        assert torch.equal(c, codes[r0:r1])
        assert torch.equal(s.view(torch.int32), scales[:, r0:r1].contiguous().view(torch.int32))
        assert total is None or torch.equal(total.nan_to_num(12345.0), tv[r0:r1].nan_to_num(12345.0))
    vd.last_error()

    pick = [r for r in [0, 1, 33, rows // 3, rows // 2, bad - 1, bad + 1, rows - 2, rows - 1] + list(range(7, rows, rows // 50)) if r != bad]
    host = lambda a: None if a is None else a.double().cpu().numpy()
    _, y = fp8.residual_rms(host(x[pick]), None if res is None else host(res[pick]), host(gamma), host(beta), 1e-6, silu)
    t = 1e-5 * (np.abs(y) + (0.0 if beta is None else np.abs(host(beta))))
    s = scales[:, pick].cpu().numpy()
    wide = s.T.astype(np.float64).repeat(128, axis=1)[:, :cols]
    byte = codes[pick].cpu().numpy()
    assert not byte[:, cols:].any()
    got = fp8.values(byte[:, :cols], np.ones_like(s), 1)
    top = np.stack([np.abs(y[:, c:c + 128]).max(1) for c in range(0, cols, 128)])
    slack = np.stack([t[:, c:c + 128].max(1) for c in range(0, cols, 128)])
    assert (np.abs(s - np.maximum(top / 448.0, 2.0 ** -126)) <= slack / 448.0 + 2.0 ** -23 * s).all()
    nearest = lambda v: np.sign(v) * fp8.E4M3[fp8.nearest_even(np.abs(v), fp8.E4M3)]
    assert (nearest((y - t) / wide) <= got).all() and (got <= nearest((y + t) / wide)).all()
