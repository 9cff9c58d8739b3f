"""8-bit operands with block scales on the GPU, through the C ABI.

What is checked, and against what (tolerances fixed before the first run):
  * quantisation: codes and scales equal the float64 oracle's (oracle/fp8.py), byte for byte, padding included, but for
    the sign of zeros; reading back equals code * scale rounded to fp32, and from there to bf16;
  * the product on operands whose every partial sum is a multiple of one unit and below 2^24 of it: exact in fp32
    whatever the order, so D equals the float64 product exactly (bf16: rounded once);
  * the product on ordinary operands: fp32 D within (K + 4 blocks + 4) 2^-23 sum |a b| (K roundings of at most one unit in the last
    place of a partial sum, in any order; per block of 128 the scales' product, the addition, and the exchange between
    parts of K) plus 2^-23 (|D| + |bias|) for alpha and the bias; bf16 D half a step, 2^-8 of the value, more;
  * the norm: the total equals the fp32 sum rounded once.  With t = 1e-5 (|y| + |beta|) every value lies between the
    quantised y - t and y + t of the oracle's y at the scale that was written, and that scale within 1e-5 of the oracle's:
    the mean of squares is off by under 70 roundings of 2^-24 (up to 64 values per lane, 8 per fp32 lane pair and vector, a tree, 32 warps), so r
    by 35, the rest by a few, SiLU by a few 2^-22 and |z| 2^-24 with |z| below 90: under 1e-5 in all.
"""
import os
import subprocess
import sys
import threading

import numpy as np
import pytest
import torch

from oracle import fp8
from patch_tiled_causal_gb300 import synth

pytestmark = pytest.mark.gpu

T = {"bf16": torch.bfloat16, "fp32": torch.float32}


@pytest.fixture(scope="module")
def vd():
    from patch_tiled_causal_gb300 import build, vaedec
    build.build()
    vaedec.load()
    vaedec.last_error()
    return vaedec


def bf16_round(a):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.float32)).to(torch.bfloat16).float().numpy()


def draw(rows, cols, seed, dt):
    """Normal values whose magnitude varies by row and by column, as an array of the type's numbers."""
    x = synth.draw_normal((rows, cols), seed) * np.exp2(np.linspace(-6, 6, rows))[:, None] * np.exp2(np.arange(cols) % 5 - 2.0)
    return bf16_round(x) if dt == "bf16" else x.astype(np.float32)


def dev(a, dt="fp32"):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.float32)).to("cuda", T[dt])


def host(codes):
    return codes.view(torch.uint8).cpu().numpy()


def no_signed_zero(byte):
    return np.where(byte == 128, 0, byte)


def filled(vd, rows, cols, block_rows):
    """Operand buffers full of other bytes."""
    codes, scales = vd.fp8_empty(rows, cols, block_rows)
    codes.view(torch.uint8).fill_(0xA5)
    scales.fill_(-7.0)
    return codes, scales


def check_operand(codes, scales, x, block_rows):
    want_c, want_s = fp8.quantize(x.astype(np.float64), block_rows)
    np.testing.assert_array_equal(scales.cpu().numpy(), want_s)
    np.testing.assert_array_equal(no_signed_zero(host(codes)), no_signed_zero(fp8.pad_codes(want_c)))
    return want_c, want_s


# ----------------------------------------------------------------------------- quantisation

SIZES = [(1, 1), (1, 16), (3, 7), (2, 130), (5, 129), (127, 128), (128, 64), (129, 257), (300, 1001), (33, 4096), (257, 384),
         (1000, 20)]


@pytest.mark.parametrize("block_rows", [1, 128])
@pytest.mark.parametrize("dt", ["bf16", "fp32"])
@pytest.mark.parametrize("rows,cols", SIZES)
def test_quantize_is_the_oracles(vd, block_rows, dt, rows, cols):
    x = draw(rows, cols, rows * 1000 + cols, dt)
    if rows > 2:
        x[1] = 0.0
        x[2, ::2] = -1e-30
    given = dev(x, dt)
    x = given.float().cpu().numpy()  # (-1e-30 is no bf16 number)
    codes, scales = filled(vd, rows, cols, block_rows)
    vd.quantize_fp8(given, codes, scales, block_rows=block_rows)
    want_c, want_s = check_operand(codes, scales, x, block_rows)
    for out in ("bf16", "fp32"):
        y = torch.full((rows, cols), 7.0, device="cuda", dtype=T[out])
        vd.dequantize_fp8(codes, scales, y, block_rows=block_rows)
        want = fp8.values(want_c, want_s, block_rows).astype(np.float32)
        np.testing.assert_array_equal(y.float().cpu().numpy(), bf16_round(want) if out == "bf16" else want)
    assert vd.last_error()[0] == vd.VAE_OK


@pytest.mark.parametrize("block_rows", [1, 128])
@pytest.mark.parametrize("dt,off,ld", [("fp32", 0, 300), ("fp32", 1, 300), ("fp32", 4, 301), ("bf16", 8, 304), ("bf16", 3, 296),
                                       ("bf16", 0, 291), ("bf16", 16, 320)])
def test_rows_of_any_stride_and_start(vd, block_rows, dt, off, ld):
    rows, cols = 140, 290
    x = draw(rows, cols, off + ld, dt)
    wide = torch.full((rows * ld + off + 64,), 3.0, device="cuda", dtype=T[dt])
    view = wide[off:off + rows * ld].view(rows, ld)[:, :cols]
    view.copy_(dev(x, dt))
    codes, scales = filled(vd, rows, cols, block_rows)
    vd.quantize_fp8(view, codes, scales, block_rows=block_rows)
    want_c, want_s = check_operand(codes, scales, x, block_rows)
    wide.fill_(3.0)
    vd.dequantize_fp8(codes, scales, view, block_rows=block_rows)
    want = fp8.values(want_c, want_s, block_rows).astype(np.float32)
    np.testing.assert_array_equal(view.float().cpu().numpy(), bf16_round(want) if dt == "bf16" else want)
    view.fill_(3.0)
    assert bool((wide == 3.0).all())  # nothing beside the matrix was written


@pytest.mark.parametrize("block_rows", [1, 128])
def test_quantize_borders(vd, block_rows):
    # every rounding border of e4m3 and its neighbours, at scales on both sides of the smallest ones
    table = fp8.E4M3
    mids = ((table[1:] + table[:-1]) / 2).astype(np.float32)
    vals = np.concatenate([mids, np.nextafter(mids, np.float32(0)), np.nextafter(mids, np.float32(500))])
    rows = []
    for s in (1.0, 1.3, 2.0 ** 100, 2.0 ** -50, 2.0 ** -69, 1.7 * 2.0 ** -69, 2.0 ** -100, 2.0 ** -126, 2.0 ** -130):
        for part in np.array_split(vals, 3):
            r = np.zeros(256, np.float32)
            r[:len(part)] = (part.astype(np.float64) * s).astype(np.float32)
            r[127] = r[255] = np.float32(-448.0 * s)
            rows.append(np.where(np.arange(256) % 3 == 1, -r, r))
    x = np.array(rows, np.float32)
    tiny = np.zeros((6, 256), np.float32)
    tiny[:, 2] = [1e-38, 1e-44, 2.0 ** -126, 3.4e38, 2.0 ** -60, np.nextafter(np.float32(2.0 ** -60), np.float32(0))]
    x = np.concatenate([x, tiny])
    if block_rows == 128:  # one row to a block: the others are zeros
        wide = np.zeros((128 * len(x), 256), np.float32)
        wide[5::128] = x
        x = wide
    codes, scales = filled(vd, len(x), 256, block_rows)
    vd.quantize_fp8(dev(x), codes, scales, block_rows=block_rows)
    check_operand(codes, scales, x, block_rows)
    assert vd.last_error()[0] == vd.VAE_OK


@pytest.mark.parametrize("block_rows", [1, 128])
@pytest.mark.parametrize("dt", ["bf16", "fp32"])
def test_quantize_flags_nan_and_infinity(vd, block_rows, dt):
    x = np.ones((300, 300), np.float32)
    x[0, 40], x[140, 299], x[299, 130] = np.nan, np.inf, -np.inf
    codes, scales = filled(vd, 300, 300, block_rows)
    vd.quantize_fp8(dev(x, dt), codes, scales, block_rows=block_rows)
    assert vd.last_error()[0] == vd.VAE_ERR_RANGE
    assert vd.last_error()[0] == vd.VAE_OK
    want_c, want_s = check_operand(codes, scales, x, block_rows)
    y = torch.empty((300, 300), device="cuda")
    vd.dequantize_fp8(codes, scales, y, block_rows=block_rows)
    np.testing.assert_array_equal(y.cpu().numpy(), fp8.values(want_c, want_s, block_rows).astype(np.float32))


def test_read_back_takes_any_codes(vd):
    byte = np.arange(256, dtype=np.uint8).repeat(2).reshape(2, 256)
    scale = np.array([[1.0, 0.0], [-3e38, 1e-45]], np.float32)
    y = torch.empty((2, 256), device="cuda")
    vd.dequantize_fp8(torch.from_numpy(byte).cuda().view(torch.float8_e4m3fn), dev(scale), y)
    with np.errstate(over="ignore"):
        np.testing.assert_array_equal(y.cpu().numpy(), fp8.values(byte, scale, 1).astype(np.float32))


@pytest.mark.parametrize("block_rows", [1, 128])
def test_offsets_past_32_bits(vd, block_rows):
    ld = 2 ** 31 + 16
    wide = torch.empty(2 * ld + 512, dtype=torch.bfloat16, device="cuda")
    view = wide.as_strided((3, 300), (ld, 1))
    x = draw(3, 300, 5, "bf16")
    view.copy_(dev(x, "bf16"))
    codes, scales = filled(vd, 3, 300, block_rows)
    vd.quantize_fp8(view, codes, scales, block_rows=block_rows)
    want_c, want_s = check_operand(codes, scales, x, block_rows)
    view.zero_()
    vd.dequantize_fp8(codes, scales, view, block_rows=block_rows)
    np.testing.assert_array_equal(view.float().cpu().numpy(), bf16_round(fp8.values(want_c, want_s, block_rows)))


# ----------------------------------------------------------------------------- the product

def operand(vd, rows, cols, block_rows, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn((rows, cols), generator=gen, device="cuda") * torch.exp2(torch.arange(cols, device="cuda") % 5 - 2.0)
    x *= torch.exp2(torch.linspace(-5, 5, rows, device="cuda"))[:, None]
    codes, scales = vd.fp8_empty(rows, cols, block_rows)
    vd.quantize_fp8(x, codes, scales, block_rows=block_rows)
    return codes, scales


def read(codes, scales, cols, block_rows):
    """Values of an operand in float64 on the GPU (torch's own reading of e4m3)."""
    s = scales.double().t().repeat_interleave(block_rows, 0)[:codes.shape[0]].repeat_interleave(128, 1)[:, :cols]
    return codes[:, :cols].double() * s


def check_product(D, a, b, M, N, K, alpha=1.0, bias=None):
    av, bv = read(*a, K, 1), read(*b, K, 128)
    want = alpha * (av @ bv.t())
    size = abs(alpha) * (av.abs() @ bv.abs().t())
    extra = want.abs()
    if bias is not None:
        want = want + bias.double()
        extra = extra + bias.double().abs()
    tol = (K + 4 * ((K + 127) // 128) + 4) * 2.0 ** -23 * size + 2.0 ** -23 * extra
    if D.dtype == torch.bfloat16:
        tol = tol + 2.0 ** -8 * (want.abs() + tol)
    over = (D.double() - want).abs() - tol
    assert bool((over <= 0).all()), (float(over.max()), int((over > 0).sum()))


PRODUCTS = [(1, 1, 1), (1, 8, 16), (1, 128, 128), (1, 1024, 1024), (2, 333, 1000), (15, 130, 31), (16, 256, 4096), (17, 256, 257),
            (32, 1000, 640), (33, 129, 33), (64, 2048, 2048), (65, 300, 129), (100, 128, 32), (128, 128, 1024), (129, 257, 1000),
            (300, 300, 300), (777, 333, 1000), (2000, 100, 129), (2500, 1100, 256), (2500, 1100, 1), (3000, 2049, 300),
            (20000, 264, 130), (256, 20000, 128), (1, 50000, 300), (64, 40001, 129), (5000, 5000, 640)]


@pytest.mark.parametrize("out", ["bf16", "fp32"])
@pytest.mark.parametrize("M,N,K", PRODUCTS)
def test_product(vd, M, N, K, out):
    a, b = operand(vd, M, K, 1, M + K), operand(vd, N, K, 128, N + K)
    D = torch.full((M, N), float("nan"), device="cuda", dtype=T[out])
    vd.gemm_fp8(*a, *b, D, K)
    check_product(D, a, b, M, N, K)
    bias = torch.randn(N, device="cuda")
    vd.gemm_fp8(*a, *b, D, K, bias=bias, alpha=-0.375)
    check_product(D, a, b, M, N, K, alpha=-0.375, bias=bias)
    again = torch.empty_like(D)
    vd.gemm_fp8(*a, *b, again, K, bias=bias, alpha=-0.375)
    assert torch.equal(D, again)  # equal calls give equal bits
    assert vd.last_error()[0] == vd.VAE_OK


@pytest.mark.parametrize("M,N,K", [(1, 200, 260), (20, 300, 1000), (50, 129, 4096), (200, 200, 700), (3000, 1030, 1000)])
def test_product_is_exact_where_fp32_is(vd, M, N, K):
    # codes -2 .. 2, scales 1/4 .. 4 per block: each sum a multiple of 2^-4 and at most K * 4 * 16 below 2^20 of it
    gen = torch.Generator(device="cuda").manual_seed(K)
    ints = lambda r: torch.randint(-2, 3, (r, (K + 15) // 16 * 16), generator=gen, device="cuda").float().to(torch.float8_e4m3fn)
    pows = lambda n: torch.exp2(torch.randint(-2, 3, ((K + 127) // 128, n), generator=gen, device="cuda").float())
    a, b = (ints(M), pows(M)), (ints(N), pows((N + 127) // 128))
    want = read(*a, K, 1) @ read(*b, K, 128).t()
    for out in ("fp32", "bf16"):
        D = torch.empty((M, N), device="cuda", dtype=T[out])
        vd.gemm_fp8(*a, *b, D, K)  # (the codes behind column K are not zeros here: they are not read)
        assert torch.equal(D, want.to(T[out]))


@pytest.mark.parametrize("M,N,K", [(5, 130, 300), (200, 130, 300), (3000, 1030, 300)])
@pytest.mark.parametrize("out,off,extra", [("bf16", 0, 2), ("bf16", 1, 1), ("bf16", 8, 6), ("fp32", 0, 2), ("fp32", 1, 3)])
def test_rows_of_d_of_any_stride_and_start(vd, M, N, K, out, off, extra):
    a, b = operand(vd, M, K, 1, 1), operand(vd, N, K, 128, 2)
    ld = N + extra
    flat = torch.full((M * ld + off + 8,), 5.0, device="cuda", dtype=T[out])
    D = flat[off:off + M * ld].view(M, ld)[:, :N]
    vd.gemm_fp8(*a, *b, D, K)
    check_product(D, a, b, M, N, K)
    D.fill_(5.0)
    assert bool((flat == 5.0).all())


@pytest.mark.parametrize("out", ["bf16", "fp32"])
@pytest.mark.parametrize("M,N,K,extra", [(20000, 1030, 130, 2), (20000, 1037, 130, 3), (9000, 3001, 260, 7)])
def test_many_tiles_whose_last_columns_fill_no_chunk(vd, M, N, K, extra, out):
    # rows of D on 16-byte boundaries, the last 16 bytes of a row not full: a warp's pieces are stored by TMA and row by
    # row in turn, tile after tile
    a, b = operand(vd, M, K, 1, 1), operand(vd, N, K, 128, 2)
    wide = torch.full((M, N + extra), 5.0, device="cuda", dtype=T[out])
    for _ in range(3):
        wide.fill_(5.0)
        vd.gemm_fp8(*a, *b, wide[:, :N], K)
        check_product(wide[:, :N], a, b, M, N, K)
        assert bool((wide[:, N:] == 5.0).all())


@pytest.mark.parametrize("M,N,K", [(3, 260, 500), (40, 260, 500), (150, 260, 500), (3000, 1100, 500)])
def test_padding_is_not_read_and_nan_stays_in_its_row(vd, M, N, K):
    a, b = operand(vd, M, K, 1, 3), operand(vd, N, K, 128, 4)
    D, E = (torch.empty((M, N), device="cuda") for _ in range(2))
    vd.gemm_fp8(*a, *b, D, K)
    for codes in (a[0], b[0]):
        codes.view(torch.uint8)[:, K:] = 0x7F  # NaN codes behind the last column
    vd.gemm_fp8(*a, *b, E, K)
    assert torch.equal(D, E)
    a[1][2, M // 2] = float("nan")    # a block of one row of A
    b[0].view(torch.uint8)[7, 9] = 0xFF  # one code of B
    b[1][1, (N - 1) // 128] = float("nan")   # the last rows of B
    vd.gemm_fp8(*a, *b, E, K)
    bad = torch.zeros((M, N), dtype=torch.bool, device="cuda")
    bad[M // 2], bad[:, 7], bad[:, (N - 1) // 128 * 128:] = True, True, True
    assert torch.equal(torch.isnan(E), bad)
    assert torch.equal(E[~bad], D[~bad])
    assert vd.last_error()[0] == vd.VAE_OK


@pytest.mark.parametrize("M,N", [(2, 130), (100, 130), (3000, 1100)])
def test_products_of_scales_that_overflow(vd, M, N):
    K = 256
    a, b = operand(vd, M, K, 1, 3), operand(vd, N, K, 128, 4)
    a[0][0, :128] = 0.0  # row 0: zeros in the block whose scales' product overflows
    a[1][0], b[1][0] = 1e30, 1e30
    D = torch.empty((M, N), device="cuda")
    vd.gemm_fp8(*a, *b, D, K)
    av, bv = read(*a, K, 1), read(*b, K, 128)
    want = (av[:1] @ bv.t()).float()
    tol = (K + 12) * 2.0 ** -23 * (av[:1].abs() @ bv.abs().t())
    assert bool(((D[:1].double() - want).abs() <= tol).all())  # zeros times infinity would be NaN


@pytest.mark.parametrize("M,N", [(2, 130), (100, 130), (3000, 1100)])
def test_signs_and_infinities_of_scales(vd, M, N):
    # operands that no quantisation writes: negative scales multiply as numbers, a product of finite scales that overflows
    # is held at the largest finite number of its sign, an infinite scale gives what its products with the sums are
    K = 128
    a, b = operand(vd, M, K, 1, 3), operand(vd, N, K, 128, 4)
    D, E = (torch.empty((M, N), device="cuda") for _ in range(2))
    vd.gemm_fp8(*a, *b, D, K)
    a[1].neg_()
    vd.gemm_fp8(*a, *b, E, K)
    assert torch.equal(E, -D)
    a[0][1] = 0.0
    a[1][0, 1], b[1][0] = -1e30, 1e30  # row 1: zeros
    vd.gemm_fp8(*a, *b, E, K)
    assert not bool(E[1].any())
    a[1][0, 1], b[1][0] = float("inf"), 1.0  # zeros times infinity
    a[1][0, 0] = float("-inf")
    vd.gemm_fp8(*a, *b, E, K)
    sums = a[0][:, :K].double() @ b[0][:, :K].double().t()
    assert bool(torch.isnan(E[1]).all())
    assert torch.equal(E[0], torch.where(sums[0] == 0, float("nan"), -torch.sign(sums[0]) * float("inf")).float())


def test_nothing_to_do(vd):
    a, b = vd.fp8_empty(0, 64), operand(vd, 128, 64, 128, 1)
    assert vd.gemm_fp8(*a, *b, torch.empty((0, 128), device="cuda"), 64).shape == (0, 128)
    vd.quantize_fp8(torch.empty((0, 64), device="cuda"), *a)
    vd.dequantize_fp8(*a, torch.empty((0, 64), device="cuda"))
    vd.residual_rmsnorm_silu_fp8(torch.empty((0, 64), device="cuda"), None, torch.ones(64, device="cuda"), None, None, *a)
    assert vd.last_error()[0] == vd.VAE_OK


# ----------------------------------------------------------------------------- the norm

def check_norm(vd, x, res, gamma, beta, eps, silu, codes, scales):
    """codes and scales against the oracle's norm, as the module's text says."""
    rows, cols = x.shape
    d = lambda a: None if a is None else a.astype(np.float64)
    _, y = fp8.residual_rms(d(x), d(res), d(gamma), d(beta), eps, silu)
    t = 1e-5 * (np.abs(y) + (0.0 if beta is None else np.abs(beta)))
    s = scales.cpu().numpy()
    byte = host(codes)
    assert not byte[:, cols:].any()
    got = fp8.values(byte[:, :cols], np.ones_like(s), 1)
    wide = s.T.astype(np.float64).repeat(128, axis=1)[:, :cols]
    top = np.stack([np.abs(y[:, c:c + 128]).max(1) for c in range(0, cols, 128)])
    slack = np.stack([t[:, c:c + 128].max(1) for c in range(0, cols, 128)])
    assert (np.abs(s - np.maximum(top / 448.0, 2.0 ** -126)) <= slack / 448.0 + 2.0 ** -23 * s).all()
    nearest = lambda v: np.sign(v) * fp8.E4M3[fp8.nearest_even(np.abs(v), fp8.E4M3)]
    lo, hi = nearest((y - t) / wide), nearest((y + t) / wide)
    assert (lo <= got).all() and (got <= hi).all()


NORMS = [(1, 1), (1, 16), (3, 7), (5, 100), (40, 128), (33, 129), (17, 256), (20, 333), (9, 512), (10, 513), (70, 1000), (65, 1024),
         (3, 1025), (6, 2048), (5, 2051), (4, 4096), (3, 6000), (2, 8192), (2, 16384), (1, 32768), (2, 32767), (1, 16385)]


@pytest.mark.parametrize("dt,rt", [("bf16", "bf16"), ("bf16", "fp32"), ("fp32", "bf16"), ("fp32", "fp32")])
@pytest.mark.parametrize("rows,cols", NORMS)
def test_norm(vd, rows, cols, dt, rt):
    x, res = draw(rows, cols, rows + cols, dt), 2 * draw(rows, cols, rows + cols + 1, rt)
    gamma = (1 + 0.2 * synth.draw_normal((cols,), 1)).astype(np.float32)
    beta = (0.1 * synth.draw_normal((cols,), 2)).astype(np.float32)
    silu = cols % 2 == 1
    codes, scales = filled(vd, rows, cols, 1)
    total = torch.full((rows, cols), 9.0, device="cuda", dtype=T[rt])
    vd.residual_rmsnorm_silu_fp8(dev(x, dt), dev(res, rt), dev(gamma), dev(beta), total, codes, scales, silu=silu)
    h = x + res  # fp32
    np.testing.assert_array_equal(total.float().cpu().numpy(), bf16_round(h) if rt == "bf16" else h)
    check_norm(vd, x, res, gamma, beta, 1e-6, silu, codes, scales)
    # without the residual, beta and the total
    codes, scales = filled(vd, rows, cols, 1)
    vd.residual_rmsnorm_silu_fp8(dev(x, dt), None, dev(gamma), None, None, codes, scales, eps=0.5, silu=not silu)
    check_norm(vd, x, None, gamma, None, 0.5, not silu, codes, scales)
    assert vd.last_error()[0] == vd.VAE_OK


@pytest.mark.parametrize("rows,cols", [(37, 120), (37, 300), (37, 1000), (7, 3001), (3, 9000)])
@pytest.mark.parametrize("dt,off,extra", [("bf16", 0, 8), ("bf16", 1, 7), ("fp32", 0, 4), ("fp32", 3, 1)])
@pytest.mark.parametrize("alias", ["none", "x", "residual"])
def test_norm_of_any_stride_and_start_and_in_place(vd, rows, cols, dt, off, extra, alias):
    x, res = draw(rows, cols, 7, dt), draw(rows, cols, 8, dt)
    gamma, beta = np.linspace(0.5, 1.5, cols).astype(np.float32), np.linspace(-1, 1, cols).astype(np.float32)
    ld = cols + extra

    def strided(a):
        flat = torch.full((rows * ld + off + 32,), 4.0, device="cuda", dtype=T[dt])
        view = flat[off:off + rows * ld].view(rows, ld)[:, :cols]
        view.copy_(dev(a, dt))
        return flat, view

    (xf, xv), (rf, rv), (tf, tv) = strided(x), strided(res), strided(np.zeros_like(x))
    if alias == "x":
        tf, tv = xf, xv
    elif alias == "residual":
        tf, tv = rf, rv
    # parameters that start off a vector boundary
    g, b = (torch.cat([torch.zeros(1, device="cuda"), dev(a)])[1:] for a in (gamma, beta))
    codes, scales = filled(vd, rows, cols, 1)
    vd.residual_rmsnorm_silu_fp8(xv, rv, g, b, tv, codes, scales)
    h = x + res
    np.testing.assert_array_equal(tv.float().cpu().numpy(), bf16_round(h) if dt == "bf16" else h)
    check_norm(vd, x, res, gamma, beta, 1e-6, False, codes, scales)
    for flat, view in ((xf, xv), (rf, rv), (tf, tv)):
        view.fill_(4.0)
        assert bool((flat == 4.0).all())


@pytest.mark.parametrize("cols", [100, 700, 5000])
def test_norm_flags_rows_it_cannot_hold(vd, cols):
    x = np.ones((5, cols), np.float32)
    x[1, cols - 1], x[2, 0], x[3, 5] = np.nan, np.inf, 1e25  # (the square of the last overflows)
    codes, scales = filled(vd, 5, cols, 1)
    total = torch.empty((5, cols), device="cuda")
    vd.residual_rmsnorm_silu_fp8(dev(x), dev(x), dev(np.ones(cols)), None, total, codes, scales)
    assert vd.last_error()[0] == vd.VAE_ERR_RANGE
    assert vd.last_error()[0] == vd.VAE_OK
    np.testing.assert_array_equal(total.cpu().numpy(), x + x)
    nan = np.isnan(scales.cpu().numpy())
    assert nan[:, 1:4].all() and not nan[:, 0].any() and not nan[:, 4].any()
    assert not host(codes)[1:4].any()
    check_norm(vd, x[[0, 4]], x[[0, 4]], np.ones(cols, np.float32), None, 1e-6, False, codes[[0, 4]], scales[:, [0, 4]])
    # an infinite parameter breaks its block of every row, and no other
    g = np.ones(cols, np.float32)
    g[3] = np.inf
    vd.residual_rmsnorm_silu_fp8(dev(np.ones((5, cols))), None, dev(g), None, None, codes, scales)
    assert vd.last_error()[0] == vd.VAE_ERR_RANGE
    np.testing.assert_array_equal(np.isnan(scales.cpu().numpy())[:, 0], np.arange(-(-cols // 128)) == 0)


def test_norm_of_zeros(vd):
    codes, scales = filled(vd, 3, 200, 1)
    z, g = torch.zeros((3, 200), device="cuda"), torch.ones(200, device="cuda")
    vd.residual_rmsnorm_silu_fp8(z, z, g, None, None, codes, scales)
    assert not no_signed_zero(host(codes)).any() and bool((scales == 2.0 ** -126).all())
    assert vd.last_error()[0] == vd.VAE_OK
    vd.residual_rmsnorm_silu_fp8(z, z, g, None, None, codes, scales, eps=0.0)  # 0 / 0
    assert vd.last_error()[0] == vd.VAE_ERR_RANGE
    assert bool(torch.isnan(scales).all())


# ----------------------------------------------------------------------------- together

def block(vd, w, x, res, gamma, bufs, total, out, stream=None):
    """One step of a residual stream: norm of the sum into an operand, and a projection of it."""
    vd.residual_rmsnorm_silu_fp8(x, res, gamma, None, total, *bufs, stream=stream)
    return vd.gemm_fp8(*bufs, *w, out, x.shape[1], stream=stream)


@pytest.mark.parametrize("rows,cols,n", [(1, 512, 512), (48, 1024, 512), (700, 1024, 1024), (3520, 512, 2048)])
def test_a_residual_stream(vd, rows, cols, n):
    # weights packed once; two blocks: the second's residual is the first's total, its input the first's projection
    wv = [torch.randn((n, cols), device="cuda") / cols ** 0.5, torch.randn((cols, n), device="cuda") / n ** 0.5]
    w = [vd.quantize_fp8(v, *vd.fp8_empty(*v.shape, 128), block_rows=128) for v in wv]
    x, res = (torch.randn((rows, cols), device="cuda", dtype=torch.bfloat16) for _ in range(2))
    res = res.float()
    gamma = torch.ones(cols, device="cuda")
    bufs, mid = vd.fp8_empty(rows, cols), vd.fp8_empty(rows, n)
    total, up = torch.empty_like(res), torch.empty((rows, n), device="cuda", dtype=torch.bfloat16)
    down = torch.empty((rows, cols), device="cuda", dtype=torch.bfloat16)
    block(vd, w[0], x, res, gamma, bufs, total, up)
    vd.quantize_fp8(up, *mid)
    vd.gemm_fp8(*mid, *w[1], down, n)
    last = torch.empty_like(res)
    vd.residual_rmsnorm_silu_fp8(down, total, gamma, None, last, *bufs, silu=True)
    got = torch.empty((rows, cols), device="cuda")
    vd.dequantize_fp8(*bufs, got)
    # each step against float64 on what it was given
    h = x.double() + res.double()
    y = h / h.square().mean(1, keepdim=True).add(1e-6).sqrt()
    assert torch.equal(total.double(), h.float().double())
    # each operand is off by half a step, 2^-4 of a value at most and 2^-4 / sqrt(3) of it in the mean; sums of independent
    # errors: relative to the product's norm, sqrt(2) 2^-4 / sqrt(3) = 0.051; the bar is half a step of both, 2^-3
    up64 = y @ wv[0].double().t()
    assert float((up.double() - up64).norm() / up64.norm()) < 2.0 ** -3
    check_product(down, mid, w[1], rows, cols, n)
    assert torch.equal(last, down.float() + total)
    h = last.double()
    y = torch.nn.functional.silu(h / h.square().mean(1, keepdim=True).add(1e-6).sqrt())
    # half a step of e4m3 at the value, or of its smallest step, 2^-10 of the scale = 2^-10 / 448 of the block's maximum
    top = torch.nn.functional.pad(y.abs(), (0, -cols % 128)).view(rows, -1, 128).amax(2).repeat_interleave(128, 1)[:, :cols]
    assert bool(((got.double() - y).abs() <= 1.0001 * (2.0 ** -4 * y.abs() + 2.0 ** -10 / 448 * top) + 1e-5).all())
    assert vd.last_error()[0] == vd.VAE_OK


@pytest.mark.parametrize("rows", [1, 40, 200, 3000])
def test_captured_and_replayed(vd, rows):
    cols = n = 1024
    w = vd.quantize_fp8(torch.randn((n, cols), device="cuda"), *vd.fp8_empty(n, cols, 128), block_rows=128)
    x, res = (torch.randn((rows, cols), device="cuda", dtype=torch.bfloat16) for _ in range(2))
    gamma, bufs = torch.ones(cols, device="cuda"), vd.fp8_empty(rows, cols)
    total, out = torch.empty_like(x), torch.empty((rows, n), device="cuda", dtype=torch.bfloat16)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):  # the first call of this size is inside the capture
        block(vd, w, x, res, gamma, bufs, total, out)
    for seed in (1, 2):
        x.copy_(torch.randn((rows, cols), generator=torch.Generator(device="cuda").manual_seed(seed), device="cuda"))
        out.zero_()
        graph.replay()
        want = block(vd, w, x, res, gamma, vd.fp8_empty(rows, cols), torch.empty_like(x), torch.empty_like(out))
        assert torch.equal(out, want)
    assert vd.last_error()[0] == vd.VAE_OK


def test_first_calls_inside_a_capture():
    """A process whose first calls of the library are captured: nothing that a capture forbids happens on the way."""
    code = """
import torch
from patch_tiled_causal_gb300 import build, vaedec as vd
build.build()
torch.cuda.init()
xs = [torch.randn((m, 512), device="cuda") for m in (1, 20, 50, 200, 3000, 1)]
xs.append(torch.randn((700, 515), device="cuda")[:, :512])
wv, gamma = torch.randn((1100, 512), device="cuda"), torch.ones(512, device="cuda")
w = vd.fp8_empty(1100, 512, 128)
bufs, outs = [vd.fp8_empty(x.shape[0], 512) for x in xs], [torch.zeros((x.shape[0], 1100), device="cuda") for x in xs]
totals = [torch.zeros((x.shape[0], 512), device="cuda") for x in xs]
backs = [torch.zeros((x.shape[0], 512), device="cuda") for x in xs]
def calls(outs, totals, backs):
    vd.quantize_fp8(wv, *w, block_rows=128)
    for x, b, o, t, y in zip(xs, bufs, outs, totals, backs):
        vd.residual_rmsnorm_silu_fp8(x, x, gamma, None, t, *b)
        vd.gemm_fp8(*b, *w, o, 512)
        vd.quantize_fp8(x, *b)
        vd.dequantize_fp8(*b, y)
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    calls(outs, totals, backs)
graph.replay()
again = [[torch.zeros_like(v) for v in l] for l in (outs, totals, backs)]
calls(*again)
torch.cuda.synchronize()
assert vd.last_error()[0] == vd.VAE_OK
for a, b in zip(outs + totals + backs, sum(again, [])):
    assert torch.equal(a, b) and bool(a.any())
print("captured first")
"""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", code], cwd=root, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "captured first" in r.stdout, r.stderr[-2000:]


def test_two_streams_and_threads(vd):
    # independent chains on streams of their own, from host threads of their own, at once
    cols, n, sizes = 1024, 1024, (1, 40, 300, 2500)
    w = vd.quantize_fp8(torch.randn((n, cols), device="cuda"), *vd.fp8_empty(n, cols, 128), block_rows=128)
    gamma = torch.ones(cols, device="cuda")
    jobs = []
    for rows in sizes:
        x, res = (torch.randn((rows, cols), device="cuda") for _ in range(2))
        out = [torch.empty((rows, n), device="cuda") for _ in range(21)]
        bufs = [vd.fp8_empty(rows, cols) for _ in range(21)]
        total = [torch.empty_like(x) for _ in range(21)]
        block(vd, w, x, res, gamma, bufs[20], total[20], out[20])
        jobs.append((x, res, bufs, total, out))
    torch.cuda.synchronize()
    errors = []

    def work(job):
        try:
            x, res, bufs, total, out = job
            stream = torch.cuda.Stream()
            for i in range(20):
                block(vd, w, x, res, gamma, bufs[i], total[i], out[i], stream=stream)
            stream.synchronize()
        except Exception as e:  # noqa: BLE001
            errors.append(e)

    threads = [threading.Thread(target=work, args=(j,)) for j in jobs]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not errors
    for x, res, bufs, total, out in jobs:
        for i in range(20):
            assert torch.equal(out[i], out[20]) and torch.equal(total[i], total[20])


def test_binding_refuses(vd):
    x = torch.zeros((8, 64), device="cuda")
    codes, scales = vd.fp8_empty(8, 64)
    w = vd.fp8_empty(16, 64, 128)
    g = torch.ones(64, device="cuda")
    bad = [lambda: vd.quantize_fp8(x, codes[:7], scales), lambda: vd.quantize_fp8(x, codes, scales[:, :7]),
           lambda: vd.quantize_fp8(x, codes, scales, block_rows=64), lambda: vd.quantize_fp8(x, codes, scales, block_rows=128),
           lambda: vd.quantize_fp8(x.half(), codes, scales), lambda: vd.quantize_fp8(x.t(), codes, scales),
           lambda: vd.quantize_fp8(x, codes.view(torch.uint8), scales), lambda: vd.quantize_fp8(x, codes, scales.double()),
           lambda: vd.gemm_fp8(codes, scales, *w, torch.empty((8, 17), device="cuda"), 64),
           lambda: vd.gemm_fp8(codes, scales, *w, torch.empty((8, 16), device="cuda"), 65),
           lambda: vd.gemm_fp8(codes, scales, *w, torch.empty((8, 16), device="cuda"), 64, bias=g),
           lambda: vd.gemm_fp8(codes, scales, codes, scales, torch.empty((8, 8), device="cuda"), 64),
           lambda: vd.residual_rmsnorm_silu_fp8(x, x[:4], g, None, None, codes, scales),
           lambda: vd.residual_rmsnorm_silu_fp8(x, x, g[:32], None, None, codes, scales),
           lambda: vd.residual_rmsnorm_silu_fp8(x, x, g, None, x.bfloat16(), codes, scales),
           lambda: vd.residual_rmsnorm_silu_fp8(x, x.cpu(), g, None, None, codes, scales)]
    for k, call in enumerate(bad):
        with pytest.raises(ValueError):
            call()
            pytest.fail(f"call {k} was taken")
    assert vd.last_error()[0] == vd.VAE_OK


def test_numbers_that_the_caller_changes_in_place(vd):
    # a call takes the value that alpha, eps, K and block_rows have then, whatever holds it
    a, b = operand(vd, 40, 256, 1, 1), operand(vd, 130, 256, 128, 2)
    alpha = torch.ones(())
    one, two = (torch.empty((40, 130), device="cuda") for _ in range(2))
    vd.gemm_fp8(*a, *b, one, torch.tensor(256), alpha=alpha)
    alpha.mul_(2.0)
    vd.gemm_fp8(*a, *b, two, np.int64(256), alpha=alpha)
    assert torch.equal(two, 2.0 * one)  # (a power of two rounds nothing)
    check_product(one, a, b, 40, 130, 256)

    x, g, eps = torch.ones((3, 256), device="cuda"), torch.ones(256, device="cuda"), torch.zeros(())
    codes, scales = vd.fp8_empty(3, 256)
    vd.residual_rmsnorm_silu_fp8(x, None, g, None, None, codes, scales, eps=eps)
    # (the mean, the root, the reciprocal and two products: a few fp32 units)
    assert torch.allclose(scales, torch.full_like(scales, 1.0 / 448.0), rtol=2.0 ** -21, atol=0.0)
    eps.fill_(3.0)  # mean of squares 1, plus 3: values of 1/2
    vd.residual_rmsnorm_silu_fp8(x, None, g, None, None, codes, scales, eps=eps)
    assert torch.allclose(scales, torch.full_like(scales, 0.5 / 448.0), rtol=2.0 ** -21, atol=0.0)

    rows = torch.tensor(1)
    vd.quantize_fp8(x, codes, scales, block_rows=rows)
    rows.fill_(128)
    with pytest.raises(ValueError):
        vd.quantize_fp8(x, codes, scales, block_rows=rows)
    wc, ws = vd.fp8_empty(3, 256, 128)
    vd.quantize_fp8(x, wc, ws, block_rows=rows)
    assert torch.equal(ws, torch.full_like(ws, 1.0 / 448.0))
    with pytest.raises(TypeError):
        vd.gemm_fp8(*a, *b, one, 256.0)
