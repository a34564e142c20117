"""The tile that a linear layer's product takes (no GPU needed)."""
import ctypes

import pytest

from cnn_cosmology_volumes_amd import cf

FWD, DX, DW, DW_ONE, DW_TWO, FWD_RES = range(6)      # dW: without an activation, with D in one part, in two


def tiles(dtype, rows, fin, fout, product):
    """(rows, columns) of the tile, splits; zeros where the kernels of few rows take it."""
    f = cf.lib().cf_internal_linear_tiles
    f.argtypes = [ctypes.c_int, ctypes.c_int64] + [ctypes.c_int32] * 3 + [ctypes.POINTER(ctypes.c_int32)]
    t = (ctypes.c_int32 * 3)()
    assert f(dtype, rows, fin, fout, product, t) == cf.CF_OK
    return tuple(t)


# us on one MI355X with tiles of 64 x 64, 128 x 128 and 256 x 128, without splits
MEASURED = {(32768, 2048, 2048): (2158, 2005, 1929), (40102, 128, 1456): (218, 205, 205), (262144, 128, 512): (485, 463, 441),
            (8192, 1024, 1024): (148, 135, 136), (32768, 512, 512): (158, 147, 141), (65536, 256, 256): (94, 87, 84),
            (4096, 2048, 2048): (276, 257, 255), (16640, 512, 256): (52, 72, 84), (262144, 64, 64): (45, 74, 71),
            (3000, 1500, 1500): (134, 190, 1e9), (32768, 1024, 128): (90, 81, 1e9), (416890, 32, 176): (191, 191, 185)}


@pytest.mark.parametrize("size", sorted(MEASURED), ids=str)
def test_fp32_takes_a_tile_near_the_fastest(size):
    """Within 4%: large products do not take the smallest tile, nor small ones the largest."""
    tm, tn, splits = tiles(cf.CF_F32, *size, FWD)
    taken = MEASURED[size][[(64, 64), (128, 128), (256, 128)].index((tm, tn))]
    assert splits == 1 and taken <= 1.04 * min(MEASURED[size])


WITH_RESIDUAL = {(40102, 128, 1456): (234, 244, 286), (32768, 512, 512): (167, 163, 162), (32768, 2048, 2048): (2157, 2017, 1956),
                 (65536, 256, 256): (94, 91, 98), (262144, 128, 512): (493, 491, 538), (8192, 1024, 1024): (155, 146, 151),
                 (7429, 333, 1001): (69, 72, 82), (20000, 700, 700): (196, 207, 211)}


@pytest.mark.parametrize("size", sorted(WITH_RESIDUAL), ids=str)
def test_fp32_with_residuals_takes_a_tile_near_the_fastest(size):
    tm, tn, splits = tiles(cf.CF_F32, *size, FWD_RES)
    taken = WITH_RESIDUAL[size][[(64, 64), (128, 128), (256, 128)].index((tm, tn))]
    assert splits == 1 and taken <= 1.04 * min(WITH_RESIDUAL[size])


def test_few_rows_take_no_tile():
    assert tiles(cf.CF_F32, 1, 2048, 2048, FWD) == (0, 0, 0) == tiles(cf.CF_BF16, 8, 512, 512, DX)
    f = cf.lib().cf_internal_linear_tiles
    assert f(cf.CF_F32, 100, 64, 64, 6, (ctypes.c_int32 * 3)()) == cf.CF_ERR_INVALID
    assert f(cf.CF_F32, 0, 64, 64, 0, (ctypes.c_int32 * 3)()) == cf.CF_ERR_INVALID


@pytest.mark.parametrize("dtype", [cf.CF_F32, cf.CF_BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("rows", [1, 3, 4, 8, 16])
def test_long_rows_are_products(rows, dtype):
    """A block of the kernels of few rows takes a whole reduction: 65536 x 1024 in bf16 was 6 times
    as long as the product.  Rows of W that would be copied first are worth it for few rows."""
    few = lambda fin, fout: tiles(dtype, rows, fin, fout, FWD) == (0, 0, 0)  # noqa: E731
    for fin in (16384, 65536):
        for fout in (16, 128, 1024, 4096, 65536):
            assert not few(fin, fout)
    assert few(512, 512) and few(2048, 2048) and few(4096, 17)
    assert few(8192, 2047) == (rows <= 4) == few(16384, 4095)
    assert not few(16384, 515)
    need = cf.cf_linear_workspace_size(dtype, rows, 65536, 1024, False)
    assert need >= 2 * 4 * rows * 1024 and need % 16 == 0      # (parts of the product's splits)


@pytest.mark.parametrize("dtype", [cf.CF_F32, cf.CF_BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("rows", [1, 4, 8, 16])
def test_wide_and_tall_backwards_are_products(rows, dtype):
    """A block of the backward of few rows takes a few rows of W over all columns: 16 x 65536 was 13 to 23 times
    as long as the products, 65536 x 16 up to 8 times."""
    few = lambda fin, fout: tiles(dtype, rows, fin, fout, DW_ONE) == (0, 0, 0) == tiles(dtype, rows, fin, fout, DX)  # noqa: E731
    for fin, fout in ((16, 16384), (16, 65536), (512, 16384), (1024, 65536), (65536, 16), (65536, 128), (2048, 16384)):
        assert not few(fin, fout)
    assert few(128, 128) and few(2048, 1024) and few(1, 1) and few(4096, 512)
    assert few(4096, 4096) == (rows <= 8) == few(4096, 2049)
    assert few(65536, 512) == (rows <= 8 and dtype == cf.CF_F32)
