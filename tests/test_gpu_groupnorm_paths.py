"""Group norm at the sizes where the library changes its way of computing
(slices held by one block, streamed samples; vectors inside a group and across
groups; rows longer than a block takes), against the definition in float64.

Tolerances: those of test_gpu_groupnorm.py."""
import numpy as np
import pytest
import torch

from cnn_cosmology_volumes_amd import cf
from gpu_util import host64, to_dev
from test_gpu_groupnorm import ACT, BF, EPS, F32, check_bwd, check_fwd, problem

pytestmark = pytest.mark.gpu

# (shape, groups)
CASES = [
    ((1, 1, 1, 2, 8), 8),             # a group of two values
    ((1, 2, 2, 2, 16), 1),            # one group of all channels
    ((4, 8, 8, 8, 32), 8),            # the most samples of the small backward
    ((5, 8, 8, 8, 32), 8),
    ((3, 8, 8, 16, 64), 32),          # groups of 2: four in a vector
    ((2, 16, 16, 16, 128), 16),       # small forward, streamed backward
    ((1, 16, 16, 17, 128), 128),      # a channel a group
    ((2, 24, 24, 24, 36), 3),         # groups of 12: across vectors of 8
    ((2, 23, 25, 27, 18), 3),         # groups of 6, odd samples
    ((1, 40, 33, 31, 6), 2),          # rows of lcm(8, 6)
    ((2, 13, 17, 19, 1032), 4),       # groups of 258
    ((1, 9, 9, 9, 2056), 257),        # 257 vectors a row
    ((1, 6, 7, 5, 4096), 16),         # the most channels
    ((7, 20, 20, 20, 48), 6),
    ((64, 4, 4, 4, 16), 4),           # many samples
]


@pytest.mark.parametrize("act,slope", [("lrelu", 0.3), ("silu", 0.0)])
@pytest.mark.parametrize("dtype", [F32, BF], ids=["f32", "bf16"])
@pytest.mark.parametrize("shape,groups", CASES, ids=["x".join(map(str, s)) + "g%d" % g for s, g in CASES])
def test_matches_oracle(shape, groups, dtype, act, slope):
    x, dy, gamma, beta = problem(shape, dtype, seed=11)
    xd, dyd, gd, bd = to_dev(x, dtype), to_dev(dy, dtype), to_dev(gamma, F32), to_dev(beta, F32)
    out = cf.cf_groupnorm_fwd(xd, groups, gd, bd, EPS, ACT[act], slope)
    check_fwd(out, x, groups, gamma, beta, act, slope, dtype)
    back = cf.cf_groupnorm_bwd(xd, dyd, groups, gd, bd, out[1], out[2], ACT[act], slope)
    check_bwd(back, x, dy, groups, gamma, beta, host64(out[1]), host64(out[2]), act, slope, dtype)


@pytest.mark.parametrize("shape,groups", [((2, 4, 4, 4, 16), 4), ((2, 30, 31, 33, 24), 3), ((2, 9, 11, 13, 515), 5)])
def test_nothing_is_read_from_the_workspace(shape, groups):
    x, dy, gamma, beta = problem(shape, BF)
    xd, dyd, gd, bd = to_dev(x, BF), to_dev(dy, BF), to_dev(gamma, F32), to_dev(beta, F32)
    got = []
    for fill in (0xFF, 0x7B):
        ws = [torch.full((max(16, cf.cf_groupnorm_workspace_size(cf.CF_BF16, shape, groups, b)),), fill, dtype=torch.uint8,
                         device="cuda") for b in (False, True)]
        f = cf.cf_groupnorm_fwd(xd, groups, gd, bd, EPS, cf.CF_ACT_SILU, ws=ws[0])
        got.append(f + cf.cf_groupnorm_bwd(xd, dyd, groups, gd, bd, f[1], f[2], cf.CF_ACT_SILU, ws=ws[1]))
    for p, q in zip(*got):
        assert torch.isfinite(p.float()).all() and torch.equal(p, q)


@pytest.mark.parametrize("shape,groups", [((2, 3, 4, 5, 24), 3), ((1, 12, 20, 16, 40), 5)])
@pytest.mark.parametrize("act", ["lrelu", "silu"])
def test_gradients_against_differences(shape, groups, act):
    """Directional derivatives of sum(y c), the forward in fp32 and summed in
    fp64.  A quotient with step h / 2 is off by a third of its change from h
    (the leaky ReLU's at slope 1, smooth) and by the rounding of y, 2^-21
    |y c| summed in squares, over h."""
    rng = np.random.default_rng(6)
    x, dy, gamma, beta = problem(shape, F32, seed=2)
    c = to_dev(dy, F32)
    p = [to_dev(v, F32) for v in (x, gamma, beta)]
    slope = 1.0

    def forward(q):
        return cf.cf_groupnorm_fwd(q[0], groups, q[1], q[2], EPS, ACT[act], slope)

    out = forward(p)
    grads = cf.cf_groupnorm_bwd(p[0], c, groups, p[1], p[2], out[1], out[2], ACT[act], slope)
    noise = 2.0 ** -21 * (out[0].double() * c.double()).norm().item()
    for k in range(3):
        d = torch.from_numpy(rng.standard_normal(p[k].shape).astype(np.float32)).cuda()

        def quotient(h):
            ends = [(forward(p[:k] + [p[k] + s * d] + p[k + 1:])[0].double() * c.double()).sum().item() for s in (h, -h)]
            return (ends[0] - ends[1]) / (2 * h)

        h = 2.0 ** -6
        wide, near = quotient(h), quotient(h / 2)
        want = (grads[k].double() * d.double()).sum().item()
        # (and the gradient's own rounding, 2^-22 of its terms in squares)
        tol = 2 * abs(wide - near) + 4 * noise / h + 2.0 ** -22 * (grads[k].double() * d.double()).norm().item() * 8
        assert abs(near - want) <= tol, (k, near, want, tol)
