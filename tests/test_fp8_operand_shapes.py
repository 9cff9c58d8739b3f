"""The binding's checks of an 8-bit operand's buffers: a buffer of the right size in another order is refused, as its numbers
would be taken for others.  No GPU: the check alone, on CPU tensors (device -1)."""
import pytest
import torch

from patch_tiled_causal_gb300 import vaedec as vd


def check(codes, scales, rows, cols, block_rows):
    assert vd._operand8(torch, codes, scales, rows, cols, block_rows, -1, "operand") == (codes.data_ptr(), scales.data_ptr())


@pytest.mark.parametrize("block_rows", [1, 128])
@pytest.mark.parametrize("rows,cols", [(1, 1), (0, 300), (3, 7), (300, 1000), (1024, 640), (128, 128)])
def test_the_documented_shapes_are_taken(rows, cols, block_rows):
    codes, scales = vd.fp8_empty(rows, cols, block_rows, device="cpu")
    check(codes, scales, rows, cols, block_rows)
    check(codes.view(-1), scales.view(-1), rows, cols, block_rows)


def test_rows_in_several_dimensions_are_taken():
    codes, scales = vd.fp8_empty(24, 300, device="cpu")
    check(codes.view(2, 3, 4, -1), scales.view(-1, 2, 3, 4), 24, 300, 1)


@pytest.mark.parametrize("rows,cols,block_rows", [(5, 300, 1), (1000, 256, 1), (300, 1000, 128), (1024, 4096, 128)])
def test_scales_by_row_blocks_first_are_refused(rows, cols, block_rows):
    codes, scales = vd.fp8_empty(rows, cols, block_rows, device="cpu")
    with pytest.raises(ValueError):
        check(codes, scales.t().contiguous(), rows, cols, block_rows)


def test_codes_of_another_shape_are_refused():
    codes, scales = vd.fp8_empty(32, 160, device="cpu")
    for shape in ((160, 32), (64, 80), (16, 320)):
        with pytest.raises(ValueError):
            check(codes.view(shape), scales, 32, 160, 1)
