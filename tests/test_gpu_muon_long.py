"""Newton-Schulz of matrices whose tiles take more threads than one launch may
have, and whose elements pass 2^31.

m rows of 2^30 values: with the exact Gram matrix (fp64) the result is Q X_0, Q
the product of the steps' m x m factors.  Rounding: 2^-21 of the terms' sizes
(three parts of bf16, fp32 sums), and of bf16 results 2^-8 of the value."""
import numpy as np
import pytest
import torch

from cnn_cosmology_volumes_amd import cf

pytestmark = pytest.mark.gpu
A, B, C, EPS = (float(np.float32(v)) for v in (3.4445, -4.7750, 2.0315, 1e-7))      # as the call takes them
CHUNK = 1 << 27


@pytest.mark.parametrize("m,dtype,steps,tall", [(1, torch.float32, 5, False), (3, torch.bfloat16, 5, False),
                                                (3, torch.bfloat16, 12, True)])
def test_long_side_of_2_to_the_30(m, dtype, steps, tall):
    n = 1 << 30
    gen = torch.Generator(device="cuda").manual_seed(m)
    x = torch.empty((n, m) if tall else (m, n), dtype=dtype, device="cuda")
    flat = x.view(-1)
    for at in range(0, flat.numel(), CHUNK):
        part = flat[at:at + CHUNK]
        part.copy_(torch.randn(part.numel(), generator=gen, device="cuda"))
    rows = (lambda at: x[at:at + CHUNK // 4].t()) if tall else (lambda at: x[:, at:at + CHUNK // 4])
    gram = torch.zeros(m, m, dtype=torch.float64, device="cuda")
    for at in range(0, n, CHUNK // 4):
        t = rows(at).double().contiguous()
        gram += torch.stack([(t * t[i]).sum(1) for i in range(m)])
    gram = gram.cpu().numpy()
    s = 1.0 / (np.sqrt(np.trace(gram)) + EPS)
    a, q = gram * s * s, np.eye(m)
    for _ in range(steps):
        p = A * np.eye(m) + B * a + C * a @ a
        q, a = p @ q, p @ a @ p
    q = torch.from_numpy(q * s).cuda()
    out = cf.cf_newton_schulz(cf.newton_schulz_params(steps, A, B, C, EPS), [x])[0]
    ours = (lambda at: out[at:at + CHUNK // 4].t()) if tall else (lambda at: out[:, at:at + CHUNK // 4])
    for at in range(0, n, CHUNK // 4):
        t, o = rows(at).double(), ours(at).double()
        for i in range(m):
            want = sum(q[i, j] * t[j] for j in range(m))
            tol = 2.0 ** -21 * sum((q[i, j] * t[j]).abs() for j in range(m))
            if dtype == torch.bfloat16:
                tol += 2.0 ** -8 * want.abs()
            assert torch.all((o[i] - want).abs() <= tol), (at, i)
