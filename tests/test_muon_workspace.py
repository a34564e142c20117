"""cf_muon's workspace is that of the path its coefficients take."""
import ctypes

import pytest

from cnn_cosmology_volumes_amd import cf


def sizes(shape, **ns):
    rows, cols = (ctypes.c_int64 * 1)(shape[0]), (ctypes.c_int64 * 1)(shape[1])
    hp = cf.muon_params(0.1, nesterov=False, ns=cf.newton_schulz_params(**ns))
    muon = cf.lib().cf_muon_workspace_size(ctypes.byref(hp), 1, rows, cols)
    return muon, cf.lib().cf_newton_schulz_workspace_size(cf.CF_F32, 1, rows, cols)


@pytest.mark.parametrize("shape", [(4096, 4096), (2500, 2048), (8000, 8192)])
def test_split_products(shape):
    """X, X^T twice, A and P at four bytes a value (rows and lines padded by
    less than a tenth here), and 134 MB of partial sums."""
    m, n = min(shape), max(shape)
    muon, most = sizes(shape)
    assert 4 * (3 * m * n + 2 * m * m) < muon < 1.1 * 4 * (3 * m * n + 2 * m * m) + (136 << 20)
    # coefficients without a small bound: five m x m buffers and U U^T's parts in fp64
    wild, same = sizes(shape, steps=2, a=20.0, b=-20.0, c=1.0)
    assert wild > 5 * 8 * m * m and same == most >= max(muon, wild)


@pytest.mark.parametrize("shape", [(108, 32), (200, 300), (128, 9000), (1, 1)])
def test_fp64_path(shape):
    muon, most = sizes(shape)
    assert muon == most == sizes(shape, steps=2, a=20.0, b=-20.0, c=1.0)[0]
