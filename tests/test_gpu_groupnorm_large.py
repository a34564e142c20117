"""Group norm of tensors past 2^31 elements: in one sample, and over samples.

Against float64, a part of the tensor at a time.  Tolerances: fp32 arithmetic,
2^-20 of the terms' sizes, and 2^-8 of bf16 values."""
import pytest
import torch

from cnn_cosmology_volumes_amd import cf

pytestmark = pytest.mark.gpu
BF = torch.bfloat16
EPS, SLOPE = 1e-5, 0.3
PART = 1 << 23      # voxels


@pytest.mark.parametrize("shape,groups", [((1, 512, 512, 512, 17), 17), ((3, 360, 368, 376, 18), 3)])
def test_past_2_to_the_31_elements(shape, groups):
    n, c, cg = shape[0], shape[-1], shape[-1] // groups
    gen = torch.Generator(device="cuda").manual_seed(1)
    x, dy = torch.empty(shape, dtype=BF, device="cuda"), torch.empty(shape, dtype=BF, device="cuda")
    assert x.numel() > 1 << 31
    for t in (x, dy):
        flat = t.view(-1)
        for at in range(0, flat.numel(), 1 << 28):
            part = flat[at:at + (1 << 28)]
            part.copy_(torch.randn(part.numel(), generator=gen, device="cuda"))
    x.view(n, -1, c).add_(0.5 * torch.arange(c, device="cuda").to(BF))
    gamma, beta = torch.rand(c, generator=gen, device="cuda") + 0.5, torch.rand(c, generator=gen, device="cuda") - 0.5
    vox = x.numel() // n // c
    parts = [(i, slice(at, min(vox, at + PART))) for i in range(n) for at in range(0, vox, PART)]
    xv, dv = x.view(n, vox, c), dy.view(n, vox, c)

    def grouped(v):                       # [n, c] sums -> the group's mean, for each channel
        return (v.view(n, groups, cg).sum(2) / (vox * cg)).repeat_interleave(cg, 1)

    s = torch.zeros(n, c, dtype=torch.float64, device="cuda")
    for i, p in parts:
        s[i] += xv[i, p].double().sum(0)
    mu = grouped(s)
    s.zero_()
    for i, p in parts:
        s[i] += (xv[i, p].double() - mu[i]).square().sum(0)
    rstd = (grouped(s) + EPS).rsqrt()
    y, m32, r32 = cf.cf_groupnorm_fwd(x, groups, gamma, beta, EPS, cf.CF_ACT_LRELU, SLOPE)
    assert torch.all((m32.double() - mu[:, ::cg]).abs() <= 2.0 ** -23 * mu[:, ::cg].abs() + 2.0 ** -40)
    assert torch.all((r32.double() / rstd[:, ::cg] - 1).abs() <= 2.0 ** -22)
    ga, be = gamma.double(), beta.double()
    yv = y.view(n, vox, c)
    for i, p in parts:
        xg = (xv[i, p].double() - mu[i]) * rstd[i] * ga
        z = xg + be
        z = torch.where(z > 0, z, SLOPE * z)
        tol = 2.0 ** -20 * (xg.abs() + be.abs()) + 2.0 ** -8 * z.abs()
        assert torch.all((yv[i, p].double() - z).abs() <= tol), (i, p)
    del y, yv
    dx, dgamma, dbeta = cf.cf_groupnorm_bwd(x, dy, groups, gamma, beta, m32, r32, cf.CF_ACT_LRELU, SLOPE)
    M, R = (t.double().repeat_interleave(cg, 1) for t in (m32, r32))

    def terms(i, p):
        h = (xv[i, p].double() - M[i]) * R[i]
        d = dv[i, p].double()
        return h, torch.where(h * ga + be > 0, d, SLOPE * d)

    a, b, size = (torch.zeros(n, c, dtype=torch.float64, device="cuda") for _ in range(3))
    for i, p in parts:
        h, d = terms(i, p)
        a[i] += d.sum(0)
        b[i] += (d * h).sum(0)
        size[i] += (d * h).square().sum(0) + d.square().sum(0)
    # roundings of the terms, 2^-22 of each, add in squares
    tol = 16 * 2.0 ** -22 * size.sum(0).sqrt()
    assert torch.all((dbeta.double() - a.sum(0)).abs() <= tol + 2.0 ** -23 * a.sum(0).abs())
    assert torch.all((dgamma.double() - b.sum(0)).abs() <= tol + 2.0 ** -23 * b.sum(0).abs())
    s1, s2 = grouped(ga * a), grouped(ga * b)
    xw = dx.view(n, vox, c)
    for i, p in parts:
        h, d = terms(i, p)
        want = R[i] * (ga * d - s1[i] - h * s2[i])
        tol = 2.0 ** -20 * R[i] * ((ga * d).abs() + s1[i].abs() + (h * s2[i]).abs()) + 2.0 ** -8 * want.abs()
        assert torch.all((xw[i, p].double() - want).abs() <= tol), (i, p)
