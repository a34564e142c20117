"""Residual joins: infinities reach what their formulas put them into, as
infinities; an offset that is not there takes no part."""
import numpy as np
import pytest
import torch

import oracle
from cnn_cosmology_volumes_amd import cf
from gpu_util import host64, to_dev

pytestmark = pytest.mark.gpu
KIND = {"rms": cf.CF_NORM_RMS, "layer": cf.CF_NORM_LAYER}


def same_kind(got, want):
    got = host64(got)
    assert np.array_equal(np.isnan(got), np.isnan(want)) and np.array_equal(np.isinf(got), np.isinf(want))
    at = np.isinf(want)
    assert np.array_equal(np.sign(got[at]), np.sign(want[at]))


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
@pytest.mark.parametrize("post", [False, True])
@pytest.mark.parametrize("c", [5, 64, 1500])
@pytest.mark.parametrize("kind", ["rms", "layer"])
def test_infinite_gates_and_gradients_without_an_offset(kind, c, post, dtype):
    rng = np.random.default_rng(c)
    shape = (2, 1, 2, 3, c)
    x, f, dr = (rng.choice([-1.5, -0.5, 0.75, 2.0], shape).astype(np.float32) for _ in range(3))
    f[..., 0] = np.float32(3.0)                          # (no centred value is 0)
    gate = rng.choice([0.5, 2.0], (2, c)).astype(np.float32)
    gpost = rng.choice([0.5, 2.0], c).astype(np.float32) if post else None
    gate[1, c // 2] = np.inf
    dev = lambda a: None if a is None else to_dev(a, torch.float32)  # noqa: E731
    with np.errstate(invalid="ignore"):
        r = oracle.resnorm_fwd(x, f, kind, 1e-5, gpost=gpost, gate=gate)[0]
    got = cf.cf_resnorm_fwd(to_dev(x, dtype), to_dev(f, dtype), KIND[kind], 1e-5, gpost=dev(gpost), gate=dev(gate),
                            need_y=False)[0]
    assert np.isinf(r[1, ..., c // 2]).all() and not np.isnan(r).any()
    same_kind(got, r)
    # an infinite gradient that reaches R
    gate[1, c // 2] = 1.0
    dr[0, 0, 1, 2, c - 1] = -np.inf
    with np.errstate(invalid="ignore"):
        want = oracle.resnorm_bwd(f, r, dr, None, kind, 1e-5, gpost=gpost, gate=gate)
    g = cf.cf_resnorm_bwd(to_dev(f, dtype), None, to_dev(dr, dtype), None, KIND[kind], 1e-5, gpost=dev(gpost), gate=dev(gate))
    assert np.isinf(want["dgate"]).sum() == 1
    same_kind(g[0], want["dx"])
    same_kind(g[1], want["df"])
    same_kind(g[6], want["dgate"])
    if post:
        same_kind(g[4], want["dgpost"])
