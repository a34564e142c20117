"""Newton-Schulz of matrices whose norm is far below eps: X_0 = x / (|x| + eps)
is small then, and each step raises it by a.  Tolerance as in test_gpu_muon.py,
relative to |X_k|: no path may lose small values."""
import numpy as np
import pytest
import torch

import oracle
from cnn_cosmology_volumes_amd import cf
from gpu_util import host64, to_dev
from test_gpu_muon import NS, bound, gradient

pytestmark = pytest.mark.gpu
F32 = torch.float32

SHAPES = [(24, 90), (64, 300), (200, 319), (530, 560), (1100, 1030)]


@pytest.mark.parametrize("eps,scale", [(1e-7, 1e-4), (1e-7, 1e-7), (1e-7, 1e-9), (1e-7, 1e-12), (1e-7, 1e-20), (1.0, 1e-6),
                                       (100.0, 1e-25)])
@pytest.mark.parametrize("shape", SHAPES, ids=["%dx%d" % s for s in SHAPES])
def test_norm_below_eps(shape, eps, scale):
    x = gradient(np.random.default_rng(3), *shape) * np.float32(scale)
    ns = NS[:4] + (eps,)
    want = oracle.newton_schulz(x, *ns)
    err = np.linalg.norm(host64(cf.cf_newton_schulz(cf.newton_schulz_params(*ns), [to_dev(x, F32)])[0]) - want)
    assert err <= bound(x, ns), (err / np.linalg.norm(want), bound(x, ns) / np.linalg.norm(want))


@pytest.mark.parametrize("ns", [(1,) + NS[1:], (2,) + NS[1:], (7,) + NS[1:], (12, 1.875, -1.25, 0.375, 1e-7),
                                (6, 0.5, 1.5, -1.0, 1e-7)])
@pytest.mark.parametrize("scale", [1e-7, 1e-12])
def test_steps_and_coefficients(ns, scale):
    x = gradient(np.random.default_rng(4), 600, 530) * np.float32(scale)
    want = oracle.newton_schulz(x, *ns)
    err = np.linalg.norm(host64(cf.cf_newton_schulz(cf.newton_schulz_params(*ns), [to_dev(x, F32)])[0]) - want)
    assert bound(x, ns) < 0.01 * np.linalg.norm(want)
    assert err <= bound(x, ns), (err, bound(x, ns))


def test_muon_of_vanishing_gradients():
    """The weight moves by lr f NewtonSchulz(u), with its rounding."""
    rng = np.random.default_rng(5)
    w0 = np.zeros((600, 530), np.float32)
    g = gradient(rng, 600, 530) * np.float32(1e-12)
    w, m = to_dev(w0, F32), torch.zeros(600, 530, device="cuda")
    cf.cf_muon(cf.muon_params(0.5, nesterov=False), [w], [to_dev(g, F32)], [m])
    want = -0.5 * oracle.newton_schulz(g, *NS)
    assert np.linalg.norm(host64(w) - want) <= 0.5 * bound(g, NS) + 2.0 ** -24 * np.linalg.norm(want)
