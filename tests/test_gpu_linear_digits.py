"""Digits of the linear layers' results: what is rounded, and how often.

Tolerances as in test_gpu_linear.py (u = 2^-24), but dX of a bf16 backward with an
activation takes D with 16 bits or more, whatever the number of rows: 2^-16 |D| of
every term of its sum, and 2^-8 of the value for dX's own type.  The SiLU of fp32 results: exp(-|z|) and the reciprocal of 1 + exp
(a step, 2 u, each), their sum and products (u each), 8 u of the value however large |z| is; its derivative
s (1 + z (1 - s)) takes both s and 1 - s so, 16 u of the sum of its terms' magnitudes."""
import numpy as np
import pytest
import torch

import oracle
from cnn_cosmology_volumes_amd import cf
from gpu_util import host64, to_dev
from test_gpu_linear import ACT, BF, F32, U, problem

pytestmark = pytest.mark.gpu


def dx_and_bound(rows, fin, fout, act, slope, seed):
    x, w, b, r, dy = problem(rows, fin, fout, BF, seed)
    pre = host64(to_dev(1.4 * np.random.default_rng(seed).standard_normal((rows, fout)), BF))
    d = dy * oracle._act(pre, act, slope)[1]
    aw = np.abs(w.astype(np.float64))
    mag = np.abs(d) @ aw.T
    e = U * (16 + 4 * np.abs(pre)) * (1 + np.abs(pre)) * np.abs(dy) if act == "silu" else U * np.abs(d)
    # D's own rounding and its two parts'; sums of 2 fout products
    tol = (e + 2.0 ** -16 * (np.abs(d) + e)) @ aw.T + (2 * fout + 2) * U * mag * 1.01
    want = d @ w.astype(np.float64).T
    tol = tol + 2.0 ** -8 * (np.abs(want) + tol)
    got = cf.cf_linear_bwd(to_dev(x, BF), to_dev(w, BF), to_dev(pre, BF), to_dev(dy, BF), ACT[act], slope)[0]
    return host64(got), want, tol


@pytest.mark.parametrize("act,slope", [("silu", 0.0), ("lrelu", 0.3), ("lrelu", 2.5)])
@pytest.mark.parametrize("rows,fin,fout", [(9, 64, 8), (15, 24, 200), (17, 5, 33), (60, 40, 24), (333, 89, 115), (700, 1024, 1032),
                                           (5000, 256, 64), (16640, 512, 256), (33001, 136, 520)])
def test_dx_takes_all_of_d(rows, fin, fout, act, slope):
    got, want, tol = dx_and_bound(rows, fin, fout, act, slope, rows)
    worst = np.max(np.abs(got - want) / tol)
    assert worst <= 1.0, worst


@pytest.mark.parametrize("rows,fin,fout", [(64, 128, 256), (2048, 512, 1024)])
def test_dx_of_a_sample_in_any_batch(rows, fin, fout):
    """Few rows keep D in fp32; the same rows in a larger batch are as near to the exact values.
    The type's rounding is up to 2^-8 of a value's power of two p, by root mean square 2^-8 p / sqrt(3);
    values spread between p and 2 p have mean squares of 7/3 p^2, and 4/3 p^2 at least where more of them
    are small: 2^-9 of the values' at most, of which D's rounding to 8 bits would take as much again."""
    got, want, tol = dx_and_bound(rows, fin, fout, "silu", 0.0, 3)
    x, w, b, r, dy = problem(rows, fin, fout, BF, 3)
    pre = host64(to_dev(1.4 * np.random.default_rng(3).standard_normal((rows, fout)), BF))
    few = host64(cf.cf_linear_bwd(to_dev(x[:8], BF), to_dev(w, BF), to_dev(pre[:8], BF), to_dev(dy[:8], BF), ACT["silu"])[0])
    rms = lambda v, at=slice(None): np.sqrt(np.mean((v[at] - want[:len(v)][at]) ** 2) / np.mean(want[:len(v)][at] ** 2))  # noqa: E731
    assert rms(few) <= 2.0 ** -9 and rms(got) <= 2.0 ** -9, (rms(few), rms(got))


@pytest.mark.parametrize("rows", [7, 16, 40, 5000])
def test_silu_of_large_arguments(rows):
    """1 x 1 layers with the weight 1: pre is X itself, and dX act' times dY."""
    rng = np.random.default_rng(rows)
    z = rng.uniform(-100, 100, (rows, 1)).astype(np.float32)
    z[0], z[1:5, 0] = -87.5, [-80.0, 88.5, -103.0, 0.0]
    dy = rng.standard_normal((rows, 1)).astype(np.float32)
    xd, w = to_dev(z, F32), torch.ones(1, 1, device="cuda")
    pre, y = cf.cf_linear_fwd(xd, w, act=ACT["silu"])
    assert torch.equal(pre, xd)
    z = z.astype(np.float64)
    s, c = 1 / (1 + np.exp(-z)), 1 / (1 + np.exp(z))
    # (e^-100 and its like are subnormal in fp32: half a step, 2^-150, in exp, times z, and in the results)
    tiny = 102 * 2.0 ** -150
    assert np.all(np.abs(host64(y) - z * s) <= 8 * U * np.abs(z * s) + tiny)
    dx = host64(cf.cf_linear_bwd(xd, w, pre, to_dev(dy, F32), ACT["silu"])[0])
    assert np.all(np.abs(dx - dy * s * (1 + z * c)) <= 16 * U * np.abs(dy) * s * (1 + np.abs(z) * c) + 5 * tiny)


def test_silu_of_infinities():
    """-inf and NaN give NaN, as -inf / (1 + exp(inf)) does; inf itself."""
    x = torch.tensor([[float("inf")], [-float("inf")], [float("nan")], [3.0]], device="cuda")
    for rows in (4, 64):
        y = cf.cf_linear_fwd(x.repeat(rows // 4, 1), torch.ones(1, 1, device="cuda"), act=ACT["silu"])[1][:, 0]
        assert torch.equal(torch.isnan(y), torch.tensor([0, 1, 1, 0], device="cuda").bool().repeat(rows // 4))
        assert bool(torch.isinf(y[0])) and bool(torch.isfinite(y[3]))
