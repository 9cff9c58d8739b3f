"""Pins of the 4-bit oracle (oracle/fp4.py): brute-force nearest values, torch's e4m3 type, layout by definition."""
import itertools

import numpy as np
import pytest
import torch

from oracle import fp4


def brute_nearest(a, table):
    """Index of the nearest entry by trying all of them; of two equally near ones the even index."""
    d = np.abs(np.asarray(a, np.float64)[..., None] - table)
    best = d.min(axis=-1, keepdims=True)
    idx = np.arange(len(table))
    even = np.where(d == best, idx + (idx % 2) * 1000, 10 ** 6).argmin(axis=-1)
    return even


def test_e4m3_table_is_torchs_type():
    want = torch.arange(127, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    np.testing.assert_array_equal(fp4.E4M3, want)
    assert torch.tensor([127], dtype=torch.uint8).view(torch.float8_e4m3fn).isnan().all()


@pytest.mark.parametrize("table", [fp4.E2M1, fp4.E4M3])
def test_nearest_even_is_the_nearest(table):
    rng = np.random.default_rng(0)
    mids = (table[1:] + table[:-1]) / 2
    a = np.concatenate([table, mids, np.nextafter(mids, 0), np.nextafter(mids, np.inf), rng.uniform(0, table[-1] * 1.2, 500)])
    np.testing.assert_array_equal(fp4.nearest_even(a, table), brute_nearest(a, table))
    bytes_ = torch.from_numpy(a[a <= 448]).float().to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    if len(table) == 127:  # (torch rounds through fp32: drop the inputs that are not fp32 numbers)
        ok = a[a <= 448] == a[a <= 448].astype(np.float32)
        np.testing.assert_array_equal(fp4.nearest_even(a[a <= 448], table)[ok], bytes_[ok])


@pytest.mark.parametrize("fmt", ["mx", "nv"])
def test_quantize_picks_the_nearest_multiple_of_its_scale(fmt):
    rng = np.random.default_rng(1)
    x = rng.standard_normal((40, 70)) * np.exp2(rng.integers(-12, 12, (40, 1)))
    x = x.astype(np.float32).astype(np.float64)
    codes, byte = fp4.quantize(x, fmt)
    s = np.repeat(fp4.scale_values(byte, fmt), fp4.BLOCK[fmt], axis=1)[:, :70]
    every = np.concatenate([fp4.E2M1, -fp4.E2M1])
    best = np.abs(x[..., None] - every * s[..., None]).min(axis=-1)
    np.testing.assert_allclose(np.abs(fp4.values(codes, byte, fmt) - x), best, rtol=1e-12, atol=0)


def test_mx_scale_rule():
    # one block per row: max|x| in [3.5, 7) 2^e
    amax = np.array([3.5, 6.999, 7.0, 4.0, 1.0, 0.875, 0.8749, 2.0 ** -126, 0.0, 2.0 ** 120])
    x = np.zeros((len(amax), 32))
    x[:, 5] = -amax
    _, byte = fp4.quantize(x, "mx")
    e = byte[:, 0].astype(int) - 127
    assert list(e) == [0, 0, 1, 0, -2, -2, -3, -127, -127, 118]
    nz = (amax > 0) & (e > -127)
    assert np.all(amax[nz] < 7 * np.exp2(e[nz])) and np.all(amax[nz] >= 3.5 * np.exp2(e[nz]))


def test_nv_scale_is_the_nearest_e4m3_and_small_blocks_vanish():
    x = np.zeros((5, 16))
    x[:, 3] = [6.0, 6.0 * 448, 6.0 * 2.0 ** -9, 6.0 * 2.0 ** -11, 6.0 * 1.0625]
    codes, byte = fp4.quantize(x, "nv")
    assert list(fp4.E4M3[byte[:, 0]]) == [1.0, 448.0, 2.0 ** -9, 0.0, 1.0]  # (1.0625 is a tie: even mantissa)
    assert list(codes[:, 3]) == [7, 7, 7, 0, 7]
    codes2, byte2 = fp4.quantize(x * 0.25, "nv", tensor_scale=0.25)
    np.testing.assert_array_equal(codes2, codes)
    np.testing.assert_array_equal(byte2, byte)


@pytest.mark.parametrize("fmt", ["mx", "nv"])
@pytest.mark.parametrize("bad", [np.nan, np.inf, -np.inf])
def test_blocks_with_nan_or_infinity_read_back_as_nan(fmt, bad):
    x = np.ones((2, 64))
    x[1, 40] = bad
    codes, byte = fp4.quantize(x, fmt)
    v = fp4.values(codes, byte, fmt)
    blk = fp4.BLOCK[fmt]
    b0 = 40 // blk * blk
    assert np.isnan(v[1, b0:b0 + blk]).all()
    v[1, b0:b0 + blk] = 1.0
    assert np.isfinite(v).all()


def test_packing_by_the_definition():
    codes = np.arange(2 * 35, dtype=np.uint8).reshape(2, 35) % 16
    p = fp4.pack_codes(codes)
    assert p.shape == (2, 32)
    for r, c in itertools.product(range(2), range(35)):
        assert (p[r, c // 2] >> (4 * (c % 2))) & 15 == codes[r, c]
    assert p[0, 17] >> 4 == 0 and not p[:, 18:].any()
    byte = np.random.default_rng(2).integers(1, 255, (131, 6)).astype(np.uint8)
    s = fp4.pack_scales(byte)
    assert s.size == 2 * 2 * 512
    # the same as axes: [row tile][4-block group][row % 32][row / 32 % 4][block % 4]
    view = s.reshape(2, 2, 32, 4, 4).transpose(0, 3, 2, 1, 4).reshape(256, 8)
    np.testing.assert_array_equal(view[:131, :6], byte)
    assert not view[131:].any() and not view[:, 6:].any()


def test_product_of_values():
    rng = np.random.default_rng(3)
    a, b = rng.standard_normal((3, 40)), rng.standard_normal((5, 40))
    got = fp4.gemm(a, b, 0.5, np.arange(5))
    for i, j in itertools.product(range(3), range(5)):
        assert abs(got[i, j] - (0.5 * sum(a[i, k] * b[j, k] for k in range(40)) + j)) < 1e-12
