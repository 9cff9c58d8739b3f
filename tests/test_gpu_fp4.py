"""Microscaled 4-bit operands on the GPU, through the C ABI.

What is checked, and against what (tolerances fixed before the first run):
  * quantisation: codes and scale bytes equal the float64 oracle's (oracle/fp4.py), byte for byte, padding included;
    reading back equals its values rounded once (twice through fp32 with a tensor scale);
  * the product on operands whose every partial sum is a multiple of one unit and below 2^24 of it: exact in
    fp32 whatever the order, so D equals the float64 product exactly (bf16: rounded once);
  * the product on ordinary operands: fp32 D within K * 2^-23 * sum |a b| (K roundings of at most one unit in
    the last place of a partial sum, in any order) plus one rounding of alpha * acc and of + bias; bf16 D half a
    step (2^-8 of the value, its rounding) more;
  * the norms: codes and scales equal the quantisation of the same norm's fp32 output (whose distance from the oracle
    other tests bound), or that of this output times 1 - 1e-5 or 1 + 1e-5: the two computations of SiLU differ by a few
    2^-22 and, in exp(-z), |z| 2^-24 of the value, under 1e-5 up to |z| = 100, and the RMS norms add up their squares in
    different orders (1024 terms in 64 or more parts: under 2^-19 of the sum).  The group norm without SiLU is
    the same arithmetic and equal bit for bit.  And every value lies within half the widest step of its block of the oracle's norm.
"""
import numpy as np
import pytest
import torch

from oracle import fp4, ops, plan
from patch_tiled_causal_gb300 import synth

pytestmark = pytest.mark.gpu

FMTS = ["mx", "nv"]


@pytest.fixture(scope="module")
def vd():
    from patch_tiled_causal_gb300 import build, vaedec
    build.build()
    vaedec.load()
    vaedec.last_error()
    return vaedec


def fid(vd, fmt):
    return vd.VAE_MXFP4 if fmt == "mx" else vd.VAE_NVFP4


def bf16_round(a):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.float32)).to(torch.bfloat16).float().numpy()


def draw(rows, cols, seed, dt):
    """Normal values whose magnitude varies by row and by column, as an array of the type's numbers."""
    x = synth.draw_normal((rows, cols), seed) * np.exp2(np.linspace(-6, 6, rows))[:, None] * np.exp2(np.arange(cols) % 5 - 2.0)
    return bf16_round(x) if dt == "bf16" else x.astype(np.float32)


def dev(a, dt):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.float32)).to("cuda", torch.bfloat16 if dt == "bf16" else torch.float32)


def upload(codes, byte):
    return torch.from_numpy(fp4.pack_codes(codes)).cuda(), torch.from_numpy(fp4.pack_scales(byte)).cuda()


# ----------------------------------------------------------------------------- quantisation

@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("dt", ["bf16", "fp32"])
@pytest.mark.parametrize("rows,cols", [(1, 1), (1, 16), (3, 7), (2, 31), (5, 33), (127, 64), (128, 128), (129, 48), (130, 200),
                                       (300, 1001), (33, 4096), (700, 256)])
def test_quantize_is_the_oracles(vd, fmt, dt, rows, cols):
    x = draw(rows, cols, rows * 1000 + cols, dt)
    if rows > 2:
        x[1] = 0.0
        x[2, ::2] = -1e-30  # rounds to a negative zero
    ts = 1.0 if fmt == "mx" else float(np.float32(np.abs(x).max() / 2688.0))
    codes, scales = vd.fp4_empty(rows, cols, fid(vd, fmt))
    codes.fill_(0xA5)
    scales.fill_(0xA5)
    vd.quantize_fp4(dev(x, dt), codes, scales, fid(vd, fmt), tensor_scale=ts)
    want_c, want_b = fp4.quantize(x.astype(np.float64), fmt, ts)
    np.testing.assert_array_equal(scales.cpu().numpy(), fp4.pack_scales(want_b))
    np.testing.assert_array_equal(codes.cpu().numpy(), fp4.pack_codes(want_c))
    for out in ("bf16", "fp32"):
        y = torch.full((rows, cols), 7.0, device="cuda", dtype=torch.bfloat16 if out == "bf16" else torch.float32)
        vd.dequantize_fp4(codes, scales, y, fid(vd, fmt), tensor_scale=ts)
        want = (fp4.values(want_c, want_b, fmt).astype(np.float32) * np.float32(ts)).astype(np.float32)
        np.testing.assert_array_equal(y.float().cpu().numpy(), bf16_round(want) if out == "bf16" else want)
    assert vd.last_error()[0] == vd.VAE_OK


@pytest.mark.parametrize("fmt", FMTS)
def test_quantize_borders(vd, fmt):
    # every rounding border of the elements, its neighbours, and block maxima around the scale's own borders
    mids = np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], np.float32)
    vals = np.concatenate([mids, np.nextafter(mids, np.float32(0)), np.nextafter(mids, np.float32(9))])
    blk = fp4.BLOCK[fmt]
    rows = []
    for top in (6.0, 6.999, 7.0, 3.5, 3.4999, 4.0, 5.3, 5.7, 6.3, 6.375, 1.0625 * 6, 1.1875 * 6):
        for s in (1.0, 1.125, 1.75, 2.0 ** -6, 2.0 ** 7):
            for part in np.array_split(vals, 2):
                r = np.zeros(blk, np.float32)
                r[:len(part)] = part * np.float32(s)
                r[-1] = -np.float32(top) * np.float32(s)
                rows.append(r)
    tiny = np.zeros((6, blk), np.float32)
    tiny[:, 2] = [1e-38, 1e-44, 2.0 ** -126, 3.3e38 if fmt == "mx" else 2000.0, 2.0 ** -11 * 6, 2.0 ** -9 * 6 * 1.4]
    x = np.concatenate([np.array(rows), tiny])
    codes, scales = vd.fp4_empty(len(x), blk, fid(vd, fmt))
    vd.quantize_fp4(torch.from_numpy(x).cuda(), codes, scales, fid(vd, fmt))
    want_c, want_b = fp4.quantize(x.astype(np.float64), fmt)
    np.testing.assert_array_equal(scales.cpu().numpy(), fp4.pack_scales(want_b))
    np.testing.assert_array_equal(codes.cpu().numpy(), fp4.pack_codes(want_c))
    assert vd.last_error()[0] == vd.VAE_OK


@pytest.mark.parametrize("fmt", FMTS)
def test_quantize_flags_what_the_format_cannot_hold(vd, fmt):
    x = np.ones((3, 96), np.float32)
    x[0, 40], x[1, 5], x[2, 95] = np.nan, np.inf, -np.inf
    codes, scales = vd.fp4_empty(3, 96, fid(vd, fmt))
    vd.quantize_fp4(torch.from_numpy(x).cuda(), codes, scales, fid(vd, fmt))
    assert vd.last_error()[0] == vd.VAE_ERR_RANGE
    assert vd.last_error()[0] == vd.VAE_OK
    want_c, want_b = fp4.quantize(x.astype(np.float64), fmt)
    np.testing.assert_array_equal(scales.cpu().numpy(), fp4.pack_scales(want_b))
    np.testing.assert_array_equal(codes.cpu().numpy(), fp4.pack_codes(want_c))
    y = torch.empty((3, 96), device="cuda")
    vd.dequantize_fp4(codes, scales, y, fid(vd, fmt))
    np.testing.assert_array_equal(np.isnan(y.cpu().numpy()), np.isnan(fp4.values(want_c, want_b, fmt)))
    if fmt == "nv":  # beyond the largest scale: clipped, and said so
        x = np.zeros((1, 16), np.float32)
        x[0, 3] = 6 * 470.0
        codes, scales = vd.fp4_empty(1, 16, vd.VAE_NVFP4)
        vd.quantize_fp4(torch.from_numpy(x).cuda(), codes, scales, vd.VAE_NVFP4)
        assert vd.last_error()[0] == vd.VAE_ERR_RANGE
        assert codes.cpu()[0, 1] == 0x70 and scales.cpu()[0] == 126
        x[0, 3:6] = [-3e38, 1e30, 1.0]  # far beyond, with a small tensor scale: the quotients would overflow
        vd.quantize_fp4(torch.from_numpy(x).cuda(), codes, scales, vd.VAE_NVFP4, tensor_scale=2.0 ** -60)
        assert vd.last_error()[0] == vd.VAE_ERR_RANGE
        assert list(codes.cpu()[0, 1:3]) == [0xF0, 0x77] and scales.cpu()[0] == 126


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("dt", ["bf16", "fp32"])
@pytest.mark.parametrize("off,pad", [(0, 8), (1, 0), (3, 5)])
def test_row_strides_and_offsets(vd, fmt, dt, off, pad):
    rows, cols = 37, 88
    x = draw(rows, cols + pad + off, 5, dt)
    wide = dev(x, dt)
    view = wide[:, off:off + cols]
    codes, scales = vd.fp4_empty(rows, cols, fid(vd, fmt))
    vd.quantize_fp4(view, codes, scales, fid(vd, fmt))
    want_c, want_b = fp4.quantize(x[:, off:off + cols].astype(np.float64), fmt)
    np.testing.assert_array_equal(codes.cpu().numpy(), fp4.pack_codes(want_c))
    np.testing.assert_array_equal(scales.cpu().numpy(), fp4.pack_scales(want_b))
    out = torch.full_like(wide, -77.0)
    vd.dequantize_fp4(codes, scales, out[:, off:off + cols], fid(vd, fmt))
    got = out.float().cpu().numpy()
    want = fp4.values(want_c, want_b, fmt).astype(np.float32)
    np.testing.assert_array_equal(got[:, off:off + cols], bf16_round(want) if dt == "bf16" else want)
    assert (got[:, :off] == -77).all() and (got[:, off + cols:] == -77).all()


def shifted(t, nbytes):
    """The same contiguous tensor at an address nbytes past a 256-byte boundary."""
    n = nbytes // t.element_size()
    buf = torch.empty(t.numel() + n + 64, dtype=t.dtype, device=t.device)
    assert buf.data_ptr() % 256 == 0
    buf[n:n + t.numel()] = t.flatten()
    return buf[n:n + t.numel()].view(t.shape)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("dt", ["bf16", "fp32"])
def test_values_on_16_byte_boundaries_only(vd, fmt, dt):
    """Inputs and outputs that start 16 bytes past a 32-byte boundary: the same bits as aligned ones."""
    f = fid(vd, fmt)
    x = dev(draw(60, 96, 15, dt), dt)
    want = vd.quantize_fp4(x, *vd.fp4_empty(60, 96, f), f)
    got = vd.quantize_fp4(shifted(x, 16), *vd.fp4_empty(60, 96, f), f)
    assert torch.equal(want[0], got[0]) and torch.equal(want[1], got[1])
    y, z = torch.empty_like(x), shifted(torch.zeros_like(x), 16)
    vd.dequantize_fp4(*want, y, f)
    vd.dequantize_fp4(*want, z, f)
    assert torch.equal(y, z)
    g, b = torch.ones(96, device="cuda"), torch.zeros(96, device="cuda")
    d = vd.gn_desc(1, 2, 5, 6, 96, 12, [0, 5], [0, 6], in_dtype=vd.VAE_FP32 if dt == "fp32" else vd.VAE_BF16)
    ws = vd.gn_workspace(d, "cuda")
    gn = [vd.patch_groupnorm_silu_fp4(t, g, b, *vd.fp4_empty(60, 96, f), ws, d, f) for t in (x, shifted(x, 16))]
    assert torch.equal(gn[0][0], gn[1][0]) and torch.equal(gn[0][1], gn[1][1])
    h = dev(draw(60, 128, 16, dt), dt)
    g, b = torch.ones(128, device="cuda"), torch.zeros(128, device="cuda")
    rms = [vd.channel_rmsnorm_silu_fp4(t, g, b, *vd.fp4_empty(60, 128, f), 1, 2, 5, 6, 128, f) for t in (h, shifted(h, 16))]
    assert torch.equal(rms[0][0], rms[1][0]) and torch.equal(rms[0][1], rms[1][1])
    vd.last_error()  # (NVFP4 with a tensor scale of 1 may clip or vanish: the bits are what is compared)


def test_quantize_offsets_beyond_32_bits(vd):
    # 4.4e9 elements (8.8 GB of bf16): the last rows come out as they do on their own
    rows, cols = 1_100_003, 4000
    x = torch.empty((rows, cols), dtype=torch.bfloat16, device="cuda")
    x.copy_(torch.linspace(-3, 3, cols, device="cuda")[None])
    tail = dev(draw(5, cols, 3, "bf16"), "bf16")
    x[-5:] = tail
    codes, scales = vd.fp4_empty(rows, cols, vd.VAE_NVFP4)
    vd.quantize_fp4(x, codes, scales, vd.VAE_NVFP4)
    c5, s5 = vd.fp4_empty(5, cols, vd.VAE_NVFP4)
    vd.quantize_fp4(tail, c5, s5, vd.VAE_NVFP4)
    assert torch.equal(codes[-5:], c5)
    assert torch.equal(codes[0], codes[rows // 2]) and torch.equal(codes[1], codes[-6])
    y5 = torch.empty_like(tail)
    vd.dequantize_fp4(c5, s5, y5, vd.VAE_NVFP4)
    x.zero_()
    vd.dequantize_fp4(codes, scales, x, vd.VAE_NVFP4)
    assert torch.equal(x[-5:], y5) and torch.equal(x[7], x[-6])


# ----------------------------------------------------------------------------- the product

def exact_operand(rows, cols, fmt, seed):
    """Random codes with scales that keep every partial product a multiple of 2^-2 (of 2^-4 in a product of two) and
    every sum of up to 4096 of them below 2^20: all partial sums are fp32 numbers."""
    rng = np.random.default_rng(seed)
    codes = rng.integers(0, 16, (rows, cols)).astype(np.uint8)
    nb = -(-cols // fp4.BLOCK[fmt])
    if fmt == "mx":
        byte = rng.integers(126, 129, (rows, nb)).astype(np.uint8)  # 1/2, 1, 2
    else:
        table = torch.tensor([0.5, 1.0, 1.5, 2.0]).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
        byte = table[rng.integers(0, 4, (rows, nb))]
    return codes, byte


SIZES = [(1, 1, 1), (1, 16, 32), (1, 1024, 1024), (2, 3, 17), (7, 33, 96), (16, 64, 4096), (17, 100, 160), (31, 200, 257), (64, 128, 128),
         (65, 129, 640), (100, 1000, 320), (127, 127, 64), (128, 128, 256), (129, 257, 288), (130, 64, 1000), (200, 512, 544),
         (256, 256, 512), (257, 300, 800), (513, 384, 768), (1000, 96, 2000), (3520, 512, 512), (5000, 1024, 1024), (300, 4096, 64)]


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("out", ["bf16", "fp32"])
@pytest.mark.parametrize("M,N,K", SIZES)
def test_gemm_exact(vd, fmt, out, M, N, K):
    ac, ab = exact_operand(M, K, fmt, 1)
    bc, bb = exact_operand(N, K, fmt, 2)
    a, b = fp4.values(ac, ab, fmt), fp4.values(bc, bb, fmt)
    tdt = torch.bfloat16 if out == "bf16" else torch.float32
    bias = np.random.default_rng(3).integers(-64, 64, N).astype(np.float32) / 4
    for bi, width in ((None, N + 3), (bias, N + 3), (bias, (N // 8 + 2) * 8)):  # rows off, and on, 16-byte boundaries
        buf = torch.full((M + 2, width), -77.0, dtype=tdt, device="cuda")  # rows behind the last, columns beside it stay
        want = fp4.gemm(a, b, 0.5, bi)
        assert np.array_equal(want, want.astype(np.float32))
        D = buf[:M, :N]
        vd.gemm_fp4(*upload(ac, ab), *upload(bc, bb), D, K, fid(vd, fmt), alpha=0.5,
                    bias=None if bi is None else torch.from_numpy(bi).cuda())
        got = buf.float().cpu().numpy()
        np.testing.assert_array_equal(got[:M, :N], bf16_round(want) if out == "bf16" else want)
        assert (got[M:] == -77).all() and (got[:, N:] == -77).all()
    dense = torch.full((M, N), -77.0, dtype=tdt, device="cuda")
    vd.gemm_fp4(*upload(ac, ab), *upload(bc, bb), dense, K, fid(vd, fmt), alpha=0.5, bias=torch.from_numpy(bias).cuda())
    assert torch.equal(dense, buf[:M, :N])
    assert vd.last_error()[0] == vd.VAE_OK


@pytest.mark.parametrize("out", ["bf16", "fp32"])
@pytest.mark.parametrize("M,N,K", [(70, 200, 512), (4000, 1000, 300)])
def test_gemm_element_aligned_bias_and_result(vd, out, M, N, K):
    """bias and D aligned to their elements only, in a frame of values that stay."""
    ac, ab = exact_operand(M, K, "nv", 21)
    bc, bb = exact_operand(N, K, "nv", 22)
    bias = (np.random.default_rng(23).integers(-64, 64, N) / 4).astype(np.float32)
    want = fp4.gemm(fp4.values(ac, ab, "nv"), fp4.values(bc, bb, "nv"), 1.0, bias)
    buf = torch.full((M + 2, N + 8), -77.0, dtype=torch.bfloat16 if out == "bf16" else torch.float32, device="cuda")
    bd = torch.zeros(N + 1, device="cuda")
    bd[1:] = torch.from_numpy(bias)
    vd.gemm_fp4(*upload(ac, ab), *upload(bc, bb), buf[1:M + 1, 1:N + 1], K, vd.VAE_NVFP4, bias=bd[1:])
    got = buf.float().cpu().numpy()
    np.testing.assert_array_equal(got[1:M + 1, 1:N + 1], bf16_round(want) if out == "bf16" else want)
    got[1:M + 1, 1:N + 1] = -77
    assert (got == -77).all()


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("out", ["bf16", "fp32"])
@pytest.mark.parametrize("M,N,K", [(1, 256, 1024), (50, 40, 96), (300, 260, 1000), (700, 512, 4096)])
def test_gemm_ordinary_operands(vd, fmt, out, M, N, K):
    xa, xb = draw(M, K, 11, "fp32"), draw(N, K, 12, "fp32")
    ta, tb = [(1.0 if fmt == "mx" else float(np.float32(np.abs(x).max() / 2688.0))) for x in (xa, xb)]
    (ac, ab), (bc, bb) = fp4.quantize(xa.astype(np.float64), fmt, ta), fp4.quantize(xb.astype(np.float64), fmt, tb)
    a, b = fp4.values(ac, ab, fmt), fp4.values(bc, bb, fmt)
    alpha = float(np.float32(ta * tb))
    bias = synth.draw_normal((N,), 13).astype(np.float32)
    want = fp4.gemm(a, b, alpha, bias)
    tol = alpha * (np.abs(a) @ np.abs(b).T) * K * 2.0 ** -23 + 2.0 ** -23 * (np.abs(want) + np.abs(bias)[None])
    if out == "bf16":
        tol = tol * (1 + 2.0 ** -8) + np.abs(want) * 2.0 ** -8
    D = torch.empty((M, N), dtype=torch.bfloat16 if out == "bf16" else torch.float32, device="cuda")
    vd.gemm_fp4(*upload(ac, ab), *upload(bc, bb), D, K, fid(vd, fmt), alpha=alpha, bias=torch.from_numpy(bias).cuda())
    err = np.abs(D.double().cpu().numpy() - want)
    assert (err <= tol).all(), (err / tol).max()


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("M,K", [(5, 200), (300, 520)])
def test_gemm_wide_scale_range_and_nan(vd, fmt, M, K):
    # scales over a wide range, one block of zeros, and a NaN block: its row is NaN, the others are untouched
    N = 70
    rng = np.random.default_rng(4)
    ac, ab = exact_operand(M, K, fmt, 5)
    bc, bb = exact_operand(N, K, fmt, 6)
    ab = rng.integers(100, 150, ab.shape).astype(np.uint8) if fmt == "mx" else rng.integers(0, 127, ab.shape).astype(np.uint8)
    ab[1, 0] = 0
    a, b = fp4.values(ac, ab, fmt), fp4.values(bc, bb, fmt)
    want = a @ b.T
    tol = (np.abs(a) @ np.abs(b).T) * K * 2.0 ** -23
    D = torch.empty((M, N), device="cuda")
    vd.gemm_fp4(*upload(ac, ab), *upload(bc, bb), D, K, fid(vd, fmt))
    assert (np.abs(D.double().cpu().numpy() - want) <= tol).all()
    ab[3, 1] = 255 if fmt == "mx" else 127
    E = torch.empty((M, N), device="cuda")
    vd.gemm_fp4(*upload(ac, ab), *upload(bc, bb), E, K, fid(vd, fmt))
    assert E[3].isnan().all()
    E[3] = D[3]
    assert torch.equal(D, E)


def test_gemm_offsets_beyond_32_bits(vd):
    # D of 4.5e9 elements (9 GB): rows of A repeat with period 1000, so must D's
    M, N, K = 1_100_000, 4096, 64
    ac, ab = exact_operand(1000, K, "mx", 7)
    bc, bb = exact_operand(N, K, "mx", 8)
    want = torch.from_numpy(fp4.gemm(fp4.values(ac, ab, "mx"), fp4.values(bc, bb, "mx"))).to(torch.bfloat16).cuda()
    codes = torch.from_numpy(fp4.pack_codes(ac)).cuda().repeat(M // 1000, 1)
    rows = torch.arange(M, device="cuda")
    byte = torch.from_numpy(ab).cuda()[rows % 1000]
    scales = torch.zeros(-(-M // 128) * 512, dtype=torch.uint8, device="cuda")
    for blk in range(2):
        scales[(rows // 128) * 512 + rows % 32 * 16 + rows % 128 // 32 * 4 + blk] = byte[:, blk]
    D = torch.empty((M, N), dtype=torch.bfloat16, device="cuda")
    vd.gemm_fp4(codes, scales, *upload(bc, bb), D, K, vd.VAE_MXFP4)
    for r in (0, 1000, 523_000, 524_000, 1_048_000, M - 1000):
        assert torch.equal(D[r:r + 1000], want), r


# ----------------------------------------------------------------------------- the norms

GN = [((1, 1, 5, 7, 64), 8, 1, 1), ((1, 3, 18, 26, 128), 32, 2, 2), ((2, 2, 9, 11, 32), 8, 3, 2), ((1, 2, 8, 16, 96), 12, 1, 3),
      ((1, 2, 24, 40, 512), 32, 1, 4), ((1, 1, 1, 1, 1024), 32, 1, 1), ((1, 1, 13, 3, 320), 8, 2, 1)]


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("dt", ["bf16", "fp32"])
@pytest.mark.parametrize("silu", [True, False])
@pytest.mark.parametrize("shape,groups,nph,npw", GN)
def test_groupnorm_fp4(vd, fmt, dt, silu, shape, groups, nph, npw):
    B, T, H, W, Cc = shape
    x = synth.draw_normal(shape, 21) * 1.5 + 0.25
    x = bf16_round(x) if dt == "bf16" else x.astype(np.float32)
    gamma, beta = (1 + 0.2 * synth.draw_normal((Cc,), 22)).astype(np.float32), (0.1 * synth.draw_normal((Cc,), 23)).astype(np.float32)
    d = vd.gn_desc(B, T, H, W, Cc, groups, plan.band_edges(H, nph), plan.band_edges(W, npw), silu=silu,
                   in_dtype=vd.VAE_FP32 if dt == "fp32" else vd.VAE_BF16, out_dtype=vd.VAE_FP32)
    ws = vd.gn_workspace(d, "cuda")
    xd, g, b = dev(x, dt), dev(gamma, "fp32"), dev(beta, "fp32")
    rows = B * T * H * W
    y = torch.empty((rows, Cc), device="cuda")
    vd.patch_groupnorm_silu(xd, g, b, y, ws, d)
    ts = 1.0 if fmt == "mx" else float(np.float32(8.0 / 2688.0))
    codes, scales = vd.fp4_empty(rows, Cc, fid(vd, fmt))
    codes.fill_(0xA5)
    scales.fill_(0xA5)
    vd.patch_groupnorm_silu_fp4(xd, g, b, codes, scales, ws, d, fid(vd, fmt), tensor_scale=ts)
    check_norm(vd, fmt, ts, y, codes, scales, not silu)
    ref = ops.group_norm(x.astype(np.float64).transpose(0, 4, 1, 2, 3), gamma, beta, groups, 1e-6)
    check_near(vd, fmt, ts, codes, scales, (ops.silu(ref) if silu else ref).transpose(0, 2, 3, 4, 1).reshape(rows, Cc))


# One launch takes frames up to 2^18 values of up to 1024 channels, three kernels the others: frames on both sides of
# each border, 1 to 512 channels per group, more frames than fit the machine at once.
GN_ROUTES = [((1, 2, 64, 64, 64), 32, 2, 2), ((1, 2, 65, 64, 64), 32, 2, 2), ((1, 1, 41, 50, 128), 8, 1, 1), ((1, 2, 40, 70, 96), 12, 2, 3),
             ((2, 1, 3, 5, 1024), 2, 1, 1), ((1, 2, 3, 5, 1280), 32, 1, 1), ((1, 1, 5, 7, 2048), 32, 1, 2), ((1, 3, 3, 11, 32), 32, 1, 1),
             ((1, 1, 1, 257, 992), 31, 1, 3), ((2, 203, 3, 3, 160), 20, 1, 1), ((1, 1, 3, 11, 1024), 1024, 1, 1)]


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("dt", ["bf16", "fp32"])
@pytest.mark.parametrize("silu", [True, False])
@pytest.mark.parametrize("shape,groups,nph,npw", GN_ROUTES)
def test_groupnorm_fp4_routes(vd, fmt, dt, silu, shape, groups, nph, npw):
    test_groupnorm_fp4(vd, fmt, dt, silu, shape, groups, nph, npw)


@pytest.mark.parametrize("centre", [0.0, 7000.0, -7000.0])
@pytest.mark.parametrize("shape,groups,npw", [((1, 2, 20, 30, 64), 64, 1), ((1, 1, 61, 70, 64), 16, 7), ((1, 1, 20, 30, 256), 8, 30)])
def test_groupnorm_fp4_large_values(vd, shape, groups, npw, centre):
    """Values near the exact sums' limit of 2^13, on both routes and to fp32.  y = a x + s with |a x|, |s| below 16: the
    roundings of a, mean, s and the result are four halves of 2^-23 of it, under 4e-6."""
    B, T, H, W, Cc = shape
    x = (centre + 900 * np.clip(synth.draw_normal(shape, 61), -1.3, 1.3)).astype(np.float32)
    d = vd.gn_desc(B, T, H, W, Cc, groups, [0, H], plan.band_edges(W, npw), silu=False, in_dtype=vd.VAE_FP32, out_dtype=vd.VAE_FP32)
    xd, g, b, ws = dev(x, "fp32"), torch.ones(Cc, device="cuda"), torch.zeros(Cc, device="cuda"), vd.gn_workspace(d, "cuda")
    rows = B * T * H * W
    y = torch.empty((rows, Cc), device="cuda")
    vd.patch_groupnorm_silu(xd, g, b, y, ws, d)
    ref = ops.group_norm(x.astype(np.float64).transpose(0, 4, 1, 2, 3), np.ones(Cc), np.zeros(Cc), groups, 1e-6)
    ref = ref.transpose(0, 2, 3, 4, 1).reshape(rows, Cc)
    assert np.abs(y.cpu().numpy() - ref).max() <= 4e-6
    codes, scales = vd.fp4_empty(rows, Cc, vd.VAE_MXFP4)
    vd.patch_groupnorm_silu_fp4(xd, g, b, codes, scales, ws, d, vd.VAE_MXFP4)
    check_norm(vd, "mx", 1.0, y, codes, scales, True)


@pytest.mark.parametrize("shape", [(1, 2, 7, 9, 64), (1, 2, 65, 64, 64)])
def test_groupnorm_fp4_range_and_repeats(vd, shape):
    """Values that the exact sums cannot hold raise the range status on both routes and stop nothing; the same call
    again, captured and replayed, and beside a copy of itself on another stream gives the same bytes."""
    B, T, H, W, Cc = shape
    rows = B * T * H * W
    d = vd.gn_desc(B, T, H, W, Cc, 8, plan.band_edges(H, 1), plan.band_edges(W, 1), silu=True, in_dtype=vd.VAE_FP32,
                   out_dtype=vd.VAE_FP32)
    x = dev(synth.draw_normal(shape, 51) * 3 - 1, "fp32")
    g, b = torch.ones(Cc, device="cuda"), torch.zeros(Cc, device="cuda")
    f = vd.VAE_MXFP4
    first = vd.patch_groupnorm_silu_fp4(x, g, b, *vd.fp4_empty(rows, Cc, f), vd.gn_workspace(d, "cuda"), d, f)
    torch.cuda.synchronize()
    for bad in (9000.0, float("nan"), float("-inf")):
        y = x.clone()
        y[0, 1, 3, 4, 5] = bad
        vd.patch_groupnorm_silu_fp4(y, g, b, *vd.fp4_empty(rows, Cc, f), vd.gn_workspace(d, "cuda"), d, f)
        torch.cuda.synchronize()
        assert vd.last_error()[0] == vd.VAE_ERR_RANGE
        assert vd.last_error()[0] == vd.VAE_OK
    side = [torch.cuda.Stream() for _ in range(2)]
    outs = [vd.fp4_empty(rows, Cc, f) for _ in range(2)]
    spaces = [vd.gn_workspace(d, "cuda") for _ in range(2)]
    graphs = []
    for o, w in zip(outs, spaces):
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            vd.patch_groupnorm_silu_fp4(x, g, b, *o, w, d, f)
    for o in outs:
        o[0].fill_(0xA5)
        o[1].fill_(0xA5)
    torch.cuda.synchronize()
    for _ in range(20):
        for gr, st in zip(graphs, side):
            with torch.cuda.stream(st):
                gr.replay()
    torch.cuda.synchronize()
    for c, s in outs:
        assert torch.equal(c, first[0]) and torch.equal(s, first[1])
    assert vd.last_error()[0] == vd.VAE_OK


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("dt", ["bf16", "fp32"])
@pytest.mark.parametrize("silu", [True, False])
@pytest.mark.parametrize("shape", [(1, 1, 1, 1, 32), (1, 1, 9, 13, 256), (2, 3, 5, 7, 64), (1, 2, 11, 12, 128), (1, 1, 7, 5, 512),
                                   (1, 2, 3, 45, 768), (1, 2, 8, 9, 1024)])
def test_rmsnorm_fp4(vd, fmt, dt, silu, shape):
    B, T, H, W, Cc = shape
    x = synth.draw_normal(shape, 31) * 2
    x = bf16_round(x) if dt == "bf16" else x.astype(np.float32)
    gamma, beta = (1 + 0.2 * synth.draw_normal((Cc,), 32)).astype(np.float32), (0.1 * synth.draw_normal((Cc,), 33)).astype(np.float32)
    xd, g, b = dev(x, dt), dev(gamma, "fp32"), dev(beta, "fp32")
    rows = B * T * H * W
    y = torch.empty((rows, Cc), device="cuda")
    vd.channel_rmsnorm_silu(xd, g, b, y, B, T, H, W, Cc, silu=silu)
    ts = 1.0 if fmt == "mx" else float(np.float32(8.0 / 2688.0))
    codes, scales = vd.fp4_empty(rows, Cc, fid(vd, fmt))
    codes.fill_(0xA5)
    scales.fill_(0xA5)
    vd.channel_rmsnorm_silu_fp4(xd, g, b, codes, scales, B, T, H, W, Cc, fid(vd, fmt), tensor_scale=ts, silu=silu)
    check_norm(vd, fmt, ts, y, codes, scales, False)
    ref = ops.channel_rms_norm(x.astype(np.float64).transpose(0, 4, 1, 2, 3), gamma, beta, 1e-6)
    check_near(vd, fmt, ts, codes, scales, (ops.silu(ref) if silu else ref).transpose(0, 2, 3, 4, 1).reshape(rows, Cc))


def check_norm(vd, fmt, ts, y, codes, scales, exact):
    f = fid(vd, fmt)
    c, s = vd.quantize_fp4(y, *vd.fp4_empty(*y.shape, f), f, tensor_scale=ts)
    if exact:
        assert torch.equal(s, scales) and torch.equal(c, codes)
    else:
        near = [(c, s)] + [vd.quantize_fp4(y * m, *vd.fp4_empty(*y.shape, f), f, tensor_scale=ts) for m in (1 - 1e-5, 1 + 1e-5)]
        assert torch.stack([scales == b for _, b in near]).any(0).all()
        got = {}
        for name, t in [("got", codes)] + [(i, a) for i, (a, _) in enumerate(near)]:
            got[name] = torch.stack((t & 15, t >> 4))
        same = torch.stack([got["got"] == got[i] for i in range(3)]).any(0)
        # where a block's scale itself lies on a border its codes belong to the other scale: few blocks
        moved = sum((b != s).sum().item() for _, b in near) * fp4.BLOCK[fmt]
        assert (~same).sum().item() <= moved
    assert vd.last_error()[0] == vd.VAE_OK


def check_near(vd, fmt, ts, codes, scales, ref):
    """Within half the widest step (4 to 6, and 6 to 7: one scale) of the block, and 1e-4 of the value for the norm itself."""
    y = torch.empty(ref.shape, device="cuda")
    vd.dequantize_fp4(codes, scales, y, fid(vd, fmt), tensor_scale=ts)
    rows, cols = ref.shape
    nb = cols // fp4.BLOCK[fmt]
    ng = -(-nb // 4)
    byte = scales.cpu().numpy().reshape(-1, ng, 32, 4, 4).transpose(0, 3, 2, 1, 4).reshape(-1, ng * 4)[:rows, :nb]
    s = np.repeat(fp4.scale_values(byte, fmt), fp4.BLOCK[fmt], axis=1) * ts
    assert (np.abs(y.double().cpu().numpy() - ref) <= s + 1e-4 * np.abs(ref) + 1e-6).all()


def test_norms_flag_range(vd):
    x = torch.ones((1, 1, 2, 2, 64), device="cuda")
    x[0, 0, 1, 1, 3] = float("nan")
    one, zero = torch.ones(64, device="cuda"), torch.zeros(64, device="cuda")
    codes, scales = vd.fp4_empty(4, 64, vd.VAE_NVFP4)
    vd.channel_rmsnorm_silu_fp4(x, one, zero, codes, scales, 1, 1, 2, 2, 64, vd.VAE_NVFP4)
    assert vd.last_error()[0] == vd.VAE_ERR_RANGE
    y = torch.empty((4, 64), device="cuda")
    vd.dequantize_fp4(codes, scales, y, vd.VAE_NVFP4)
    assert y[3].isnan().all() and not y[:3].isnan().any()


# ----------------------------------------------------------------------------- used together

@pytest.mark.parametrize("fmt", FMTS)
def test_norm_product_chain(vd, fmt):
    """The attention's projections on 4-bit operands: weights packed once, group norm into an operand, q, k and v
    from it; captured into a graph, replayed on new inputs, on a stream of its own, and two graphs in turn."""
    B, T, H, W, Cc = 1, 2, 10, 14, 256
    rows = B * T * H * W
    f = fid(vd, fmt)
    gamma, beta = (1 + 0.2 * synth.draw_normal((Cc,), 41)).astype(np.float32), (0.1 * synth.draw_normal((Cc,), 42)).astype(np.float32)
    ws_ = [synth.draw_normal((Cc, Cc), 43 + i).astype(np.float32) / 16 for i in range(3)]
    biases = [synth.draw_normal((Cc,), 46 + i).astype(np.float32) for i in range(3)]
    tw = [1.0 if fmt == "mx" else float(np.float32(np.abs(w).max() / 2688.0)) for w in ws_]
    tx = 1.0 if fmt == "mx" else float(np.float32(8.0 / 2688.0))
    packed = []
    for w, t in zip(ws_, tw):
        c, s = vd.fp4_empty(Cc, Cc, f)
        packed.append(vd.quantize_fp4(dev(w, "fp32"), c, s, f, tensor_scale=t))
    d = vd.gn_desc(B, T, H, W, Cc, 32, [0, 4, 10], [0, 14], silu=False, in_dtype=vd.VAE_BF16)

    def program():
        st = {"x": torch.zeros((B, T, H, W, Cc), dtype=torch.bfloat16, device="cuda"), "op": vd.fp4_empty(rows, Cc, f),
              "ws": vd.gn_workspace(d, "cuda"),
              "out": [torch.empty((rows, Cc), dtype=torch.bfloat16, device="cuda") for _ in range(3)]}

        def step():
            vd.patch_groupnorm_silu_fp4(st["x"], g, b, *st["op"], st["ws"], d, f, tensor_scale=tx)
            for i in range(3):
                vd.gemm_fp4(*st["op"], *packed[i], st["out"][i], Cc, f, bias=bias[i], alpha=tx * tw[i])
        return st, step

    g, b, bias = dev(gamma, "fp32"), dev(beta, "fp32"), [dev(v, "fp32") for v in biases]
    xs = [bf16_round(synth.draw_normal((B, T, H, W, Cc), 50 + i)) for i in range(2)]

    def want(x, i):
        y = ops.group_norm(x.astype(np.float64).transpose(0, 4, 1, 2, 3), gamma, beta, 32, 1e-6).transpose(0, 2, 3, 4, 1)
        qa, qw = fp4.quantize(y.reshape(rows, Cc), fmt, tx), fp4.quantize(ws_[i].astype(np.float64), fmt, tw[i])
        return fp4.gemm(fp4.values(*qa, fmt, tx), fp4.values(*qw, fmt, tw[i]), 1.0, biases[i])

    eager = []
    side = torch.cuda.Stream()
    progs = [program(), program()]
    for (st, step), x in zip(progs, xs):
        st["x"].copy_(dev(x, "bf16"))
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            step()
        torch.cuda.current_stream().wait_stream(side)
        eager.append([o.clone() for o in st["out"]])
    for outs, x in zip(eager, xs):
        for i in range(3):
            r = want(x, i)
            # a norm value next to a rounding border may go the other way (fp32 against float64): a few codes of a
            # row, each at most one step; relative L2 well under the rounding of bf16 outputs
            e = outs[i].double().cpu().numpy() - r
            assert np.linalg.norm(e) <= 2.0 ** -8 * np.linalg.norm(r)
    graphs = []
    for st, step in progs:
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            step()
        graphs.append(gr)
    for st, _ in progs:
        for o in st["out"]:
            o.zero_()
    for k in range(3):
        for gr in graphs:
            gr.replay()
    torch.cuda.synchronize()
    for (st, _), outs in zip(progs, eager):
        for o, e in zip(st["out"], outs):
            assert torch.equal(o, e)
    progs[0][0]["x"].copy_(dev(xs[1], "bf16"))  # new inputs in the first graph's buffers
    graphs[0].replay()
    torch.cuda.synchronize()
    for o, e in zip(progs[0][0]["out"], eager[1]):
        assert torch.equal(o, e)
    assert vd.last_error()[0] == vd.VAE_OK


def test_two_streams_at_once(vd):
    """Products and quantisations on two streams side by side, many times: nothing is shared between calls."""
    f = vd.VAE_NVFP4
    sets = []
    for i, (M, N, K) in enumerate([(3000, 512, 512), (40, 300, 1500)]):
        ac, ab = exact_operand(M, K, "nv", 60 + i)
        bc, bb = exact_operand(N, K, "nv", 70 + i)
        want = torch.from_numpy(fp4.gemm(fp4.values(ac, ab, "nv"), fp4.values(bc, bb, "nv"))).float().cuda()
        x = dev(draw(700 + 13 * i, 1000 + 7 * i, 80 + i, "fp32"), "fp32")
        op = vd.quantize_fp4(x, *vd.fp4_empty(*x.shape, f), f)
        sets.append({"a": upload(ac, ab), "b": upload(bc, bb), "K": K, "want": want, "D": [torch.zeros_like(want) for _ in range(4)],
                     "x": x, "op": [t.clone() for t in op], "out": vd.fp4_empty(*x.shape, f), "s": torch.cuda.Stream()})
    torch.cuda.synchronize()
    for k in range(40):
        for s in sets:
            vd.gemm_fp4(*s["a"], *s["b"], s["D"][k % 4], s["K"], f, stream=s["s"])
            vd.quantize_fp4(s["x"], *s["out"], f, stream=s["s"])
    torch.cuda.synchronize()
    for s in sets:
        for d in s["D"]:
            assert torch.equal(d, s["want"])
        assert torch.equal(s["out"][0], s["op"][0]) and torch.equal(s["out"][1], s["op"][1])
    assert vd.last_error()[0] == vd.VAE_OK


def test_a_pending_range_fault_stops_no_later_call(vd):
    """A flagged block (NaN) of an earlier call, not yet asked for, and long and short products and a conv after it: whole
    results, and the flag still there afterwards."""
    f = vd.VAE_MXFP4
    x = torch.full((4, 64), float("nan"), device="cuda")
    vd.quantize_fp4(x, *vd.fp4_empty(4, 64, f), f)
    for M, N, K in ((2000, 600, 3000), (9, 70, 4096)):
        ac, ab = exact_operand(M, K, "mx", 90)
        bc, bb = exact_operand(N, K, "mx", 91)
        D = torch.zeros((M, N), device="cuda")
        vd.gemm_fp4(*upload(ac, ab), *upload(bc, bb), D, K, f)
        np.testing.assert_array_equal(D.cpu().numpy(), fp4.gemm(fp4.values(ac, ab, "mx"), fp4.values(bc, bb, "mx")))
    a = torch.ones((3000, 4096), dtype=torch.bfloat16, device="cuda")
    b = torch.ones((512, 4096), dtype=torch.bfloat16, device="cuda")
    E = torch.zeros((3000, 512), device="cuda")
    vd.gemm_bf16(a, b, E)
    assert (E == 4096).all()
    assert vd.last_error()[0] == vd.VAE_ERR_RANGE
    assert vd.last_error()[0] == vd.VAE_OK


def test_first_calls_inside_a_capture():
    """A process whose first calls of the library are captured: nothing that a capture forbids happens on the way."""
    code = """
import torch
from patch_tiled_causal_gb300 import vaedec as vd
x = torch.randn(300, 256, device="cuda", dtype=torch.bfloat16)
one, zero = torch.ones(256, device="cuda"), torch.zeros(256, device="cuda")
f = vd.VAE_NVFP4
q, r, g = (vd.fp4_empty(300, 256, f) for _ in range(3))
D, E = torch.zeros(300, 300, device="cuda"), torch.zeros(300, 300, device="cuda")
d = vd.gn_desc(1, 1, 15, 20, 256, 32, [0, 15], [0, 20])
ws = vd.gn_workspace(d, "cuda")
y = torch.empty(300, 256, device="cuda")
torch.cuda.synchronize()
gr = torch.cuda.CUDAGraph()
with torch.cuda.graph(gr):
    vd.quantize_fp4(x, *q, f)
    vd.channel_rmsnorm_silu_fp4(x, one, zero, *r, 1, 1, 15, 20, 256, f)
    vd.patch_groupnorm_silu_fp4(x, one, zero, *g, ws, d, f)
    vd.gemm_fp4(*q, *r, D, 256, f)
    vd.gemm_fp4(*g, *r, E, 256, f)
    vd.dequantize_fp4(*g, y, f)
gr.replay()
torch.cuda.synchronize()
d1, e1, y1 = D.clone(), E.clone(), y.clone()
D.zero_(), E.zero_(), y.zero_()
vd.gemm_fp4(*q, *r, D, 256, f)
vd.gemm_fp4(*g, *r, E, 256, f)
vd.dequantize_fp4(*g, y, f)
assert torch.equal(D, d1) and torch.equal(E, e1) and torch.equal(y, y1) and D.abs().sum() > 0 and E.abs().sum() > 0
assert vd.last_error()[0] == vd.VAE_OK
print("captured first")
"""
    import os
    import subprocess
    import sys
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", code], cwd=root, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "captured first" in r.stdout, r.stderr[-2000:]


def test_binding_checks(vd):
    codes, scales = vd.fp4_empty(8, 64, vd.VAE_MXFP4)
    x = torch.zeros((8, 64), device="cuda")
    with pytest.raises(ValueError):
        vd.quantize_fp4(x.t(), codes, scales, vd.VAE_MXFP4)  # columns not adjacent
    with pytest.raises(ValueError):
        vd.quantize_fp4(x.half(), codes, scales, vd.VAE_MXFP4)
    with pytest.raises(ValueError):
        vd.quantize_fp4(torch.zeros((9, 64), device="cuda"), codes, scales, vd.VAE_MXFP4)  # codes too small
    with pytest.raises(ValueError):
        vd.quantize_fp4(x, codes, scales[:256], vd.VAE_MXFP4)
    with pytest.raises(ValueError):
        vd.quantize_fp4(x, codes.cpu(), scales, vd.VAE_MXFP4)
    with pytest.raises(ValueError):
        vd.gemm_fp4(codes, scales, codes, scales, torch.zeros((8, 8), device="cuda"), 128, vd.VAE_MXFP4)
    with pytest.raises(ValueError):
        vd.gemm_fp4(codes, scales, codes, scales, torch.zeros((8, 8), device="cuda"), 64, vd.VAE_MXFP4, bias=torch.zeros(7, device="cuda"))
    with pytest.raises(ValueError):
        vd.gemm_fp4(codes, scales, codes, scales, torch.zeros((1, 8), device="cuda").expand(8, 8), 64, vd.VAE_MXFP4)
    with pytest.raises(vd.VaeError):
        vd.quantize_fp4(x, codes, scales, vd.VAE_MXFP4, tensor_scale=2.0)
    empty = torch.empty((0, 64), device="cuda")
    vd.quantize_fp4(empty, *vd.fp4_empty(0, 64, vd.VAE_MXFP4), vd.VAE_MXFP4)
    vd.gemm_fp4(*vd.fp4_empty(0, 64, vd.VAE_MXFP4), codes, scales, torch.empty((0, 8), device="cuda"), 64, vd.VAE_MXFP4)
    assert vd.last_error()[0] == vd.VAE_OK


# ----------------------------------------------------------------------------- more channels than a block has vectors

# 257 to 768 vectors of 8 channels: whole, uneven and nearly empty slices of them, groups inside and across slices
GN_WIDE = [((1, 2, 3, 5, 2080), 260, 1, 1), ((1, 1, 5, 7, 2080), 520, 2, 3), ((1, 1, 4, 3, 2112), 33, 1, 2), ((2, 1, 3, 5, 4096), 1024, 1, 1),
           ((1, 1, 3, 5, 4128), 3, 1, 1), ((1, 1, 7, 9, 6144), 32, 2, 2), ((1, 2, 1, 1, 6144), 768, 1, 1)]


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("dt", ["bf16", "fp32"])
@pytest.mark.parametrize("shape,groups,nph,npw", GN_WIDE)
def test_groupnorm_fp4_wide(vd, fmt, dt, shape, groups, nph, npw):
    test_groupnorm_fp4(vd, fmt, dt, dt == "bf16", shape, groups, nph, npw)


@pytest.mark.parametrize("dt", ["bf16", "fp32"])
@pytest.mark.parametrize("shape,groups,nph,npw", GN_WIDE + [((1, 1, 4, 5, 2056), 257, 1, 1)])
def test_groupnorm_wide(vd, dt, shape, groups, nph, npw):
    """The wider outputs' group norm, fp32 out and no SiLU: y = a x + s with a = rstd gamma, s = beta - mean a.  Each of mean,
    rstd, a, mean a, s and y is rounded once (half a step, 2^-24): 3 roundings of a x, 6 of mean a and 2 of beta at most.
    The statistics take x in steps of 2^-18: the mean moves by 2^-19 at most, the deviation likewise."""
    B, T, H, W, Cc = shape
    x = synth.draw_normal(shape, 71) * 1.5 + 0.25
    x = bf16_round(x) if dt == "bf16" else x.astype(np.float32)
    gamma, beta = (1 + 0.2 * synth.draw_normal((Cc,), 72)).astype(np.float32), (0.1 * synth.draw_normal((Cc,), 73)).astype(np.float32)
    d = vd.gn_desc(B, T, H, W, Cc, groups, plan.band_edges(H, nph), plan.band_edges(W, npw), silu=False,
                   in_dtype=vd.VAE_FP32 if dt == "fp32" else vd.VAE_BF16, out_dtype=vd.VAE_FP32)
    y = torch.full(shape, float("nan"), device="cuda")
    vd.patch_groupnorm_silu(dev(x, dt), dev(gamma, "fp32"), dev(beta, "fp32"), y, vd.gn_workspace(d, "cuda"), d)
    g = x.astype(np.float64).reshape(B, T, H, W, groups, Cc // groups)
    mean, var = g.mean((2, 3, 5), keepdims=True), g.var((2, 3, 5), keepdims=True)
    a = np.broadcast_to(1 / np.sqrt(var + 1e-6), g.shape).reshape(shape) * gamma
    mean, dev_ = np.broadcast_to(mean, g.shape).reshape(shape), np.broadcast_to(np.sqrt(var + 1e-6), g.shape).reshape(shape)
    want = (x - mean) * a + beta
    tol = 6 * 2.0 ** -24 * (np.abs(a * x) + np.abs(a * mean) + np.abs(beta)) + 2.0 ** -19 * np.abs(a) + 2.0 ** -19 / dev_ * np.abs(want - beta)
    err = np.abs(y.cpu().numpy() - want)
    assert (err <= tol).all(), (err / tol).max()
    assert vd.last_error()[0] == vd.VAE_OK


@pytest.mark.parametrize("out", ["bf16", "fp32"])
@pytest.mark.parametrize("K", [256, 512, 1024, 2048])
def test_gemm_ragged_columns_in_every_cluster_size(vd, out, K):
    """Last tiles whose columns end inside a lane's 4, K in 1, 2, 4 and 8 parts: the lanes of a warp store differently, and
    all of them are back together before the cluster's CTAs leave.  Many calls in a row, into rows on and off 16 bytes."""
    tdt = torch.bfloat16 if out == "bf16" else torch.float32
    for N in (1, 2, 3, 5, 63, 126, 129, 255):
        M = 131 if N == 129 else 5
        ac, ab = exact_operand(M, K, "nv", 100 + N)
        bc, bb = exact_operand(N, K, "nv", 200 + N)
        want = torch.from_numpy(fp4.gemm(fp4.values(ac, ab, "nv"), fp4.values(bc, bb, "nv"))).to(tdt).cuda()
        a, b = upload(ac, ab), upload(bc, bb)
        for ld in (N, (N + 7) // 8 * 8):
            buf = torch.full((20, M, ld), -77.0, dtype=tdt, device="cuda")
            for i in range(20):
                vd.gemm_fp4(*a, *b, buf[i, :, :N], K, vd.VAE_NVFP4)
            assert (buf[:, :, :N] == want).all() and (buf[:, :, N:] == -77).all()
    assert vd.last_error()[0] == vd.VAE_OK


# ----------------------------------------------------------------------------- group norm of many frames

def launches(call):
    """Kernels, copies and clears that a call enqueues, counted in a graph that captures it."""
    import ctypes
    gr = torch.cuda.CUDAGraph(keep_graph=True)
    with torch.cuda.graph(gr):
        call()
    n = ctypes.c_size_t(0)
    assert ctypes.CDLL("libcuda.so.1").cuGraphGetNodes(ctypes.c_void_p(gr.raw_cuda_graph()), None, ctypes.byref(n)) == 0
    return n.value


@pytest.mark.parametrize("shape", [(1, 1, 3, 3, 160), (2, 150, 3, 3, 160), (1, 3, 32, 64, 128), (1, 77, 18, 26, 128)])
def test_groupnorm_fp4_one_launch_for_few_frames_only(vd, shape):
    """One launch per call only where every frame's 8 blocks are on the GPU at once (152 SMs, two blocks each: 38 frames at
    most); more frames wait for each other there (400 of 3 x 3 x 160: 65 us against 14)."""
    B, T, H, W, Cc = shape
    rows, f = B * T * H * W, vd.VAE_NVFP4
    d = vd.gn_desc(B, T, H, W, Cc, Cc // 8, [0, H], [0, W])
    x, ws = torch.randn(shape, device="cuda").to(torch.bfloat16), vd.gn_workspace(d, "cuda")
    g, b, op = torch.ones(Cc, device="cuda"), torch.zeros(Cc, device="cuda"), vd.fp4_empty(rows, Cc, f)

    def call():
        vd.patch_groupnorm_silu_fp4(x, g, b, *op, ws, d, f, tensor_scale=2.0 ** -7)

    call()
    assert (launches(call) == 1) == (B * T <= 38)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("dt", ["bf16", "fp32"])
@pytest.mark.parametrize("shape", [(1, 32, 3, 7, 64), (4, 9, 2, 5, 128), (1, 37, 3, 7, 64), (3, 13, 2, 5, 96), (1, 1300, 1, 3, 32)])
def test_groupnorm_fp4_frame_counts(vd, fmt, dt, shape):
    """Frames up to, at and beyond what fits the machine at once."""
    test_groupnorm_fp4(vd, fmt, dt, dt == "fp32", shape, shape[-1] // 8, 1, 2)


# ----------------------------------------------------------------------------- the product on many tiles
# More than 152 tiles of 128 x 128 run as CTA pairs on 256 x 256 tiles: more k blocks than stages, K that ends inside a block,
# after each of a k block's four steps, and several tiles per pair.

PAIRS = [(2600, 1024, 1300), (2500, 1030, 2000), (5100, 1100, 1600), (2561, 1025, 4096), (2570, 1290, 1330), (2600, 1000, 2320),
         (20000, 130, 1545), (700, 4000, 1409)]


def takes_pairs(M, N):
    return -(-M // 128) * -(-N // 128) > 152


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("out", ["bf16", "fp32"])
@pytest.mark.parametrize("M,N,K", PAIRS)
def test_pairs_exact(vd, fmt, out, M, N, K):
    assert takes_pairs(M, N)
    test_gemm_exact(vd, fmt, out, M, N, K)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("out", ["bf16", "fp32"])
@pytest.mark.parametrize("M,N,K", [(2600, 1000, 1300), (2500, 1100, 2080), (5000, 1024, 96)])
def test_pairs_ordinary_operands(vd, fmt, out, M, N, K):
    assert takes_pairs(M, N)
    test_gemm_ordinary_operands(vd, fmt, out, M, N, K)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("K", [520, 1544])
def test_pairs_wide_scale_range_and_nan(vd, fmt, K):
    """Scales over a wide range in A and B, a block of zeros, and a NaN block in each: a row and a column of NaN, nothing
    else moves."""
    M, N = 2600, 1030
    assert takes_pairs(M, N)
    rng = np.random.default_rng(14)
    (ac, ab), (bc, bb) = exact_operand(M, K, fmt, 15), exact_operand(N, K, fmt, 16)
    lo, hi = (100, 150) if fmt == "mx" else (0, 127)
    ab, bb = [rng.integers(lo, hi, t.shape).astype(np.uint8) for t in (ab, bb)]
    ab[1, 0] = 0
    a, b = fp4.values(ac, ab, fmt), fp4.values(bc, bb, fmt)
    want, tol = a @ b.T, (np.abs(a) @ np.abs(b).T) * K * 2.0 ** -23
    D = torch.empty((M, N), device="cuda")
    vd.gemm_fp4(*upload(ac, ab), *upload(bc, bb), D, K, fid(vd, fmt))
    assert (np.abs(D.double().cpu().numpy() - want) <= tol).all()
    nan = 255 if fmt == "mx" else 127
    ab[2000, 1], bb[777, -1] = nan, nan
    E = torch.empty((M, N), device="cuda")
    vd.gemm_fp4(*upload(ac, ab), *upload(bc, bb), E, K, fid(vd, fmt))
    assert E[2000].isnan().all() and E[:, 777].isnan().all()
    E[2000], E[:, 777] = D[2000], D[:, 777]
    assert torch.equal(D, E)


def test_pairs_on_two_streams_in_graphs_and_after_a_range_fault(vd):
    """Two long products on two streams at once, launched and replayed, with a flagged block of an earlier call pending."""
    f = vd.VAE_NVFP4
    vd.quantize_fp4(torch.full((4, 64), float("inf"), device="cuda"), *vd.fp4_empty(4, 64, f), f)
    sets = []
    for i, (M, N, K) in enumerate([(5000, 600, 1700), (2600, 1030, 2100)]):
        assert takes_pairs(M, N)
        (ac, ab), (bc, bb) = exact_operand(M, K, "nv", 160 + i), exact_operand(N, K, "nv", 170 + i)
        want = torch.from_numpy(fp4.gemm(fp4.values(ac, ab, "nv"), fp4.values(bc, bb, "nv"))).float().cuda()
        sets.append({"op": upload(ac, ab) + upload(bc, bb), "K": K, "want": want, "D": [torch.zeros_like(want) for _ in range(3)],
                     "s": torch.cuda.Stream()})
    torch.cuda.synchronize()
    for k in range(30):
        for s in sets:
            vd.gemm_fp4(*s["op"], s["D"][k % 2], s["K"], f, stream=s["s"])
    torch.cuda.synchronize()
    for s in sets:
        s["g"] = torch.cuda.CUDAGraph()
        with torch.cuda.graph(s["g"]):
            vd.gemm_fp4(*s["op"], s["D"][2], s["K"], f)
    for k in range(30):
        for s in sets:
            with torch.cuda.stream(s["s"]):
                s["g"].replay()
    torch.cuda.synchronize()
    for s in sets:
        for d in s["D"]:
            assert torch.equal(d, s["want"])
    assert vd.last_error()[0] == vd.VAE_ERR_RANGE
    assert vd.last_error()[0] == vd.VAE_OK
