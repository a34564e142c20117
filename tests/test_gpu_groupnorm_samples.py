"""Group norm of small volumes over many samples: held beside each other in a
block, one to a block with the joining launch, and streamed.

Tolerances: those of test_gpu_groupnorm.py."""
import pytest
import torch

from cnn_cosmology_volumes_amd import cf
from gpu_util import host64, to_dev
from test_gpu_groupnorm import ACT, BF, EPS, F32, check_bwd, check_fwd, problem

pytestmark = pytest.mark.gpu

# (shape, groups)
CASES = [
    ((16, 2, 2, 2, 24), 3),           # sixteen samples in a block
    ((6, 4, 4, 4, 64), 8),
    ((200, 1, 1, 4, 8), 4),
    ((512, 1, 1, 8, 4), 2),           # a thread a sample, and too few threads
    ((513, 1, 1, 8, 4), 2),
    ((260, 2, 2, 2, 6), 2),           # more than 256 blocks of whole rows
    ((300, 1, 1, 3, 16), 2),
    ((40, 3, 3, 3, 12), 4),
    ((9, 7, 5, 3, 160), 32),
    ((12, 8, 8, 8, 256), 32),         # wider slices
    ((24, 12, 12, 12, 128), 32),      # too many narrow slices
    ((8, 12, 12, 12, 128), 32),
]


@pytest.mark.parametrize("act,slope", [("lrelu", 0.3), ("silu", 0.0)])
@pytest.mark.parametrize("dtype", [F32, BF], ids=["f32", "bf16"])
@pytest.mark.parametrize("shape,groups", CASES, ids=["x".join(map(str, s)) + "g%d" % g for s, g in CASES])
def test_matches_oracle(shape, groups, dtype, act, slope):
    x, dy, gamma, beta = problem(shape, dtype, seed=12)
    xd, dyd, gd, bd = to_dev(x, dtype), to_dev(dy, dtype), to_dev(gamma, F32), to_dev(beta, F32)
    out = cf.cf_groupnorm_fwd(xd, groups, gd, bd, EPS, ACT[act], slope)
    check_fwd(out, x, groups, gamma, beta, act, slope, dtype)
    back = cf.cf_groupnorm_bwd(xd, dyd, groups, gd, bd, out[1], out[2], ACT[act], slope)
    check_bwd(back, x, dy, groups, gamma, beta, host64(out[1]), host64(out[2]), act, slope, dtype)


@pytest.mark.parametrize("shape,groups", [((16, 2, 2, 2, 24), 3), ((8, 8, 8, 8, 64), 8)])
def test_nothing_is_read_from_the_workspace_and_replays(shape, groups):
    x, dy, gamma, beta = problem(shape, BF)
    xd, dyd, gd, bd = to_dev(x, BF), to_dev(dy, BF), to_dev(gamma, F32), to_dev(beta, F32)
    _, mean, rstd = cf.cf_groupnorm_fwd(xd, groups, gd, bd, EPS, cf.CF_ACT_SILU)
    nbytes = cf.cf_groupnorm_workspace_size(cf.CF_BF16, shape, groups, True)
    got = []
    for fill in (0xFF, 0x7B):
        ws = torch.full((max(16, nbytes),), fill, dtype=torch.uint8, device="cuda")
        got.append(cf.cf_groupnorm_bwd(xd, dyd, groups, gd, bd, mean, rstd, cf.CF_ACT_SILU, ws=ws))
    for p, q in zip(*got):
        assert torch.isfinite(p.float()).all() and torch.equal(p, q)
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        out = cf.cf_groupnorm_bwd(xd, dyd, groups, gd, bd, mean, rstd, cf.CF_ACT_SILU)
    for seed in (3, 4, 5):
        dyd.copy_(to_dev(problem(shape, BF, seed=seed)[1], BF))
        want = cf.cf_groupnorm_bwd(xd, dyd, groups, gd, bd, mean, rstd, cf.CF_ACT_SILU)
        graph.replay()
        torch.cuda.synchronize()
        for p, q in zip(out, want):
            assert torch.equal(p, q)
