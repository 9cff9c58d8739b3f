"""The float64 oracle of the 8-bit operands with block scales (oracle/fp8.py) against definitions written another way."""
import numpy as np
import pytest
import torch

from oracle import fp8

# every finite non-negative e4m3 value, from torch's own type
TABLE = torch.arange(127, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()


def test_table_of_values():
    byte = np.arange(256, dtype=np.uint8)[None]
    got = fp8.values(byte, np.ones((2, 1), np.float32), 1)[0]
    want = torch.arange(256, dtype=torch.int32).to(torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    np.testing.assert_array_equal(got, want)


@pytest.mark.parametrize("block_rows", [1, 128])
@pytest.mark.parametrize("rows,cols", [(1, 1), (3, 130), (129, 128), (130, 257)])
def test_every_value_is_the_nearest_multiple_of_its_scale(rows, cols, block_rows):
    x = (np.random.default_rng(rows + cols).standard_normal((rows, cols)) * np.exp2(np.arange(cols) % 7 - 3.0)).astype(np.float32)
    byte, scale = fp8.quantize(x.astype(np.float64), block_rows)
    assert scale.shape == (-(-cols // 128), -(-rows // block_rows))
    for rb in range(scale.shape[1]):
        for cb in range(scale.shape[0]):
            part = x[rb * block_rows:(rb + 1) * block_rows, cb * 128:(cb + 1) * 128]
            got = byte[rb * block_rows:(rb + 1) * block_rows, cb * 128:(cb + 1) * 128]
            s = np.float32(np.abs(part).max() / np.float32(448.0))
            assert scale[cb, rb] == s
            q = np.abs((part / s).astype(np.float32).astype(np.float64))
            far = np.abs(q[..., None] - TABLE)
            np.testing.assert_array_equal(np.abs(q - TABLE[got & 127]), far.min(-1))
            assert TABLE[got & 127].max() == 448.0
            np.testing.assert_array_equal(got >= 128, part < 0)


def test_ties_go_to_the_even_code_and_torch_agrees():
    mids = (TABLE[1:] + TABLE[:-1]) / 2
    x = np.zeros((1, 128 * 2))
    x[0, :63], x[0, 127] = mids[:63], 448.0  # the scale is 1
    x[0, 128:128 + 63], x[0, 255] = mids[63:], -448.0
    byte, scale = fp8.quantize(x, 1)
    np.testing.assert_array_equal(scale, 1.0)
    np.testing.assert_array_equal(byte[x == 0] & 127, 0)
    assert not np.any(byte[0, :63] & 1) and not np.any(byte[0, 128:128 + 63] & 1)
    np.testing.assert_array_equal(byte, torch.from_numpy(x).to(torch.float8_e4m3fn).view(torch.uint8).numpy())


def test_tiny_zero_and_broken_blocks():
    x = np.zeros((4, 128))
    x[1, 3], x[1, 4] = 1e-40, -2e-42
    x[2, 5], x[3, 6] = np.nan, -np.inf
    byte, scale = fp8.quantize(x, 1)
    assert scale[0, 0] == scale[0, 1] == np.float32(2.0 ** -126)
    v = fp8.values(byte, scale, 1)
    assert abs(v[1, 3] - 1e-40) <= 2.0 ** -136 and abs(v[1, 4] + 2e-42) <= 2.0 ** -136  # half of e4m3's 2^-9
    assert np.isnan(scale[0, 2:]).all() and not byte[2:].any() and np.isnan(v[2:]).all()


def test_product_and_norm():
    rng = np.random.default_rng(3)
    a, b, bias = rng.standard_normal((3, 5)), rng.standard_normal((4, 5)), rng.standard_normal(4)
    want = np.array([[sum(a[i, k] * b[j, k] for k in range(5)) * 0.5 + bias[j] for j in range(4)] for i in range(3)])
    np.testing.assert_allclose(fp8.gemm(a, b, 0.5, bias), want, rtol=1e-13)
    g = rng.standard_normal(5)
    h, y = fp8.residual_rms(a, 2 * a, g, None, 0.25, True)
    np.testing.assert_array_equal(h, a + 2 * a)
    ref = torch.nn.functional.rms_norm(torch.from_numpy(3 * a), (5,), torch.from_numpy(g), 0.25)
    np.testing.assert_allclose(y, torch.nn.functional.silu(ref).numpy(), rtol=1e-12)
    np.testing.assert_allclose(fp8.residual_rms(a, None, g, bias[:1].repeat(5), 0.0, False)[1],
                               torch.nn.functional.rms_norm(torch.from_numpy(a), (5,), torch.from_numpy(g), 0.0).numpy() + bias[0],
                               rtol=1e-12)
