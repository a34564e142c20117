"""The tile that a linear layer's product takes (no GPU needed)."""
import ctypes

import pytest

from cnn_cosmology_volumes_amd import cf

FWD, DX, DW, DW_ONE, DW_TWO = range(5)      # dW: without an activation, with D in one part, in two


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


def test_few_rows_take_no_tile():
    assert tiles(cf.CF_F32, 1, 2048, 2048, FWD) == (0, 0, 0) == tiles(cf.CF_BF16, 8, 512, 512, DX)
    f = cf.lib().cf_internal_linear_tiles
    assert f(cf.CF_F32, 100, 64, 64, 5, (ctypes.c_int32 * 3)()) == cf.CF_ERR_INVALID
    assert f(cf.CF_F32, 0, 64, 64, 0, (ctypes.c_int32 * 3)()) == cf.CF_ERR_INVALID
