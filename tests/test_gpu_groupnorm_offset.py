"""Group norm of values whose mean is far above their spread: x - mean is taken
with all of the mean's digits, not with its fp32 rounding.

Tolerances as in test_gpu_groupnorm.py without its term of the mean's rounding
(u |mean| rstd |gamma|, 1e-3 here): with mu the fp32 mean and d = mean - mu,
  z = (x - mu) (rstd gamma) + (beta - d rstd gamma)
has relative errors of x - mu, the product and the sum, 4u |xhat gamma|, u |beta|,
and of d's terms (each u |mean| rstd |gamma| at most) 8 u^2 |mean| rstd |gamma|;
all doubled.  rstd's own error, 2^-44 (max |x| rstd)^2, is that of sums of x^2."""
import numpy as np
import pytest

import oracle
from cnn_cosmology_volumes_amd import cf
from gpu_util import host64, to_dev
from test_gpu_groupnorm import ACT, EPS, F32, U, per_element, problem

pytestmark = pytest.mark.gpu

CASES = [((1, 5, 5, 5, 8), 2), ((2, 8, 8, 8, 256), 32), ((2, 3, 3, 5, 7), 7),      # one launch
         ((1, 40, 41, 42, 8), 2), ((2, 31, 17, 29, 60), 12), ((2, 9, 11, 13, 515), 5),
         ((1, 13, 17, 19, 4096), 4096)]                                            # streamed, the most groups


@pytest.mark.parametrize("act,slope", [("lrelu", 1.0), ("silu", 0.0)])
@pytest.mark.parametrize("offset", [1e2, -1e3, 3e4])
@pytest.mark.parametrize("shape,groups", CASES, ids=["x".join(map(str, s)) + "g%d" % g for s, g in CASES])
def test_forward(shape, groups, offset, act, slope):
    x, _, gamma, beta = problem(shape, F32, offset=offset)
    y, mo, ro = oracle.groupnorm_fwd(x, groups, gamma, beta, EPS, act, slope)
    got, mean, rstd = cf.cf_groupnorm_fwd(to_dev(x, F32), groups, to_dev(gamma, F32), to_dev(beta, F32), EPS, ACT[act],
                                          slope)
    big = np.abs(x.reshape(shape[0], -1, groups, shape[-1] // groups)).max(axis=(1, 3)).astype(np.float64)
    assert np.all(np.abs(host64(mean) - mo) <= U * np.abs(mo) + 2.0 ** -45 * big)
    f = x.reshape(shape[0], -1, shape[-1]).astype(np.float64)
    M, R, B = (per_element(v, shape, groups) for v in (mo, ro, big))
    xg = (f - M) * R * gamma
    z = xg + beta
    ez = 2 * U * (4 * np.abs(xg) + np.abs(beta)) + 16 * U * U * np.abs(M) * R * np.abs(gamma)
    ez = ez + np.abs(xg) * 2.0 ** -44 * (B * R) ** 2 + 2.0 ** -45 * B * R * np.abs(gamma)
    tol = 1.1 * ez + U * (8 + 2 * np.abs(z)) * np.abs(y.reshape(f.shape))
    err = np.abs(host64(got).reshape(f.shape) - y.reshape(f.shape))
    assert np.all(err <= tol + 1e-37), float((err / (tol + 1e-37)).max())
