"""The group-norm oracle against central differences of its own forward, and
the entry points' refusals (validation happens before any GPU work, so these
run without a GPU; pointers passed here are never dereferenced)."""
import ctypes

import numpy as np
import pytest
import torch

import oracle
from cnn_cosmology_volumes_amd import cf

FAKE = ctypes.c_void_p(0x100000)
MIS = ctypes.c_void_p(0x100008)


@pytest.mark.parametrize("act", ["lrelu", "silu"])
def test_backward_is_the_forwards_derivative(act):
    rng = np.random.default_rng(5)
    shape, groups, eps, slope = (2, 3, 2, 2, 6), 3, 1e-3, 0.3
    x, dy = rng.standard_normal(shape) + 0.5, rng.standard_normal(shape)
    gamma, beta = rng.uniform(0.5, 1.5, 6), rng.uniform(-0.5, 0.5, 6)
    f = lambda a, g, b: float((oracle.groupnorm_fwd(a, groups, g, b, eps, act, slope)[0] * dy).sum())
    _, mean, rstd = oracle.groupnorm_fwd(x, groups, gamma, beta, eps, act, slope)
    dx, dg, db = oracle.groupnorm_bwd(x, dy, groups, gamma, beta, mean, rstd, act, slope)
    # central differences: truncation h^2 f"/6 and cancellation 2^-52 |f| / h, both below 1e-8 here, beside
    # the leaky ReLU's kink, which no sampled point lies within 1e-4 of
    z = (oracle.groupnorm_fwd(x, groups, gamma, beta, eps, "lrelu", 1.0)[0])
    assert np.abs(z).min() > 1e-4
    h = 1e-5
    for i in rng.choice(x.size, 12, replace=False):
        e = np.zeros(x.size)
        e[i] = h
        e = e.reshape(shape)
        assert abs((f(x + e, gamma, beta) - f(x - e, gamma, beta)) / (2 * h) - dx.flat[i]) < 1e-6
    for c in range(6):
        e = np.eye(6)[c] * h
        assert abs((f(x, gamma + e, beta) - f(x, gamma - e, beta)) / (2 * h) - dg[c]) < 1e-6
        assert abs((f(x, gamma, beta + e) - f(x, gamma, beta - e)) / (2 * h) - db[c]) < 1e-6


def test_one_group_per_channel_is_instance_norm():
    rng = np.random.default_rng(6)
    x = rng.standard_normal((1, 3, 4, 5, 7))
    g, b = rng.standard_normal(7), rng.standard_normal(7)
    y, _, _ = oracle.groupnorm_fwd(x, 7, g, b, 1e-5, "lrelu", 1.0)
    yb, _, _ = oracle.batchnorm_fwd(x, g, b, 1e-5)      # one sample: the same statistics
    assert np.allclose(y, yb, rtol=1e-12, atol=1e-12)


def _fwd(dt=cf.CF_BF16, shape=(2, 64, 64, 64, 64), groups=16, eps=1e-5, act=cf.CF_ACT_LRELU, slope=0.3, X=FAKE, ws=FAKE,
         wsb=1 << 30, gamma=FAKE):
    return cf.lib().cf_groupnorm_fwd(dt, cf.dims(shape), X, groups, gamma, FAKE, eps, act, slope, FAKE, FAKE, FAKE, ws,
                                     wsb, None)


def _bwd(dt=cf.CF_F32, shape=(2, 64, 64, 64, 64), groups=16, act=cf.CF_ACT_SILU, slope=0.0, dY=FAKE, ws=FAKE,
         wsb=1 << 30):
    return cf.lib().cf_groupnorm_bwd(dt, cf.dims(shape), FAKE, dY, groups, FAKE, FAKE, FAKE, FAKE, act, slope, FAKE,
                                     FAKE, FAKE, ws, wsb, None)


def test_refusals():
    inv, uns, wse = cf.CF_ERR_INVALID, cf.CF_ERR_UNSUPPORTED, cf.CF_ERR_WORKSPACE
    assert _fwd(dt=5) == inv
    assert _fwd(shape=(0, 4, 4, 4, 8), groups=2) == inv
    assert _fwd(shape=(1, 0, 4, 4, 8), groups=2) == inv
    assert _fwd(groups=0) == inv and _fwd(groups=-1) == inv and _fwd(groups=7) == inv
    assert b"groups" in cf.lib().cf_last_error()
    assert _fwd(eps=0.0) == inv and _fwd(eps=float("nan")) == inv and _fwd(eps=float("inf")) == inv
    assert _fwd(act=2) == inv and _fwd(slope=-0.1) == inv and _fwd(slope=float("nan")) == inv
    assert _fwd(X=None) == inv and _fwd(X=MIS) == inv and _fwd(gamma=None) == inv
    assert _fwd(shape=(1, 2, 2, 2, 8192), groups=2) == uns
    assert _fwd(shape=(70000, 1, 1, 1, 8), groups=2) == uns
    assert _fwd(wsb=16) == wse and _fwd(ws=None) == inv
    assert _bwd(dY=None) == inv and _bwd(dY=MIS) == inv and _bwd(wsb=16) == wse and _bwd(groups=3) == inv
    assert _bwd(act=-1) == inv


def test_workspace_sizes():
    size = cf.cf_groupnorm_workspace_size
    # small groups are held in registers: no workspace
    assert size(cf.CF_BF16, (1, 4, 4, 4, 256), 32, False) == 0
    assert size(cf.CF_F32, (2, 8, 8, 8, 256), 32, True) == 0
    # streaming: partial sums, far below the tensor's own size
    for bwd in (False, True):
        n = size(cf.CF_BF16, (8, 128, 128, 128, 32), 8, bwd)
        assert 0 < n < 8 * 128 ** 3 * 32 * 2 // 64
    assert size(cf.CF_BF16, (1, 4, 4, 4, 256), 3, False) == 0       # invalid


def test_binding_refuses_other_layouts():
    x = torch.zeros(1, 2, 2, 2, 8)
    v = torch.zeros(8)
    with pytest.raises(ValueError):
        cf.cf_groupnorm_fwd(x.transpose(1, 4), 2, torch.zeros(2), torch.zeros(2), 1e-5)
    with pytest.raises(ValueError):
        cf.cf_groupnorm_fwd(x, 2, torch.zeros(7), v, 1e-5)
    with pytest.raises(TypeError):
        cf.cf_groupnorm_fwd(x, 2, v.double(), v, 1e-5)
    with pytest.raises(TypeError):
        cf.cf_groupnorm_fwd(x.half(), 2, v, v, 1e-5)
    m = torch.zeros(1, 2)
    with pytest.raises(TypeError):
        cf.cf_groupnorm_bwd(x, x.bfloat16(), 2, v, v, m, m)
    with pytest.raises(ValueError):
        cf.cf_groupnorm_bwd(x, x[:, :1].contiguous(), 2, v, v, m, m)


@pytest.mark.parametrize("dt,shape,groups", [(cf.CF_BF16, (8, 8, 8, 8, 64), 8), (cf.CF_F32, (16, 8, 8, 8, 256), 32)])
def test_sums_of_samples_need_their_workspace(dt, shape, groups):
    n = cf.cf_groupnorm_workspace_size(dt, shape, groups, True)
    assert n >= 16 * shape[0] * shape[4]
    assert _bwd(dt=dt, shape=shape, groups=groups, wsb=n - 1) == cf.CF_ERR_WORKSPACE
    assert _bwd(dt=dt, shape=shape, groups=groups, ws=None) == cf.CF_ERR_INVALID
