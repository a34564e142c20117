"""GPU parity of the Newton-Schulz products (cf_newton_schulz) and Muon's
update (cf_muon) against the fp64 oracle.

Tolerance.  A step computed with products of relative error e per operand and
term adds at most e K |X_k| to X_{k+1} in the Frobenius norm, K = |a| + 2 |b| +
4 |c| (the operands of each of the three products are within 1.3 of unit
norm), and later steps raise it by at most |a| each, the slope at 0:
  |out - exact| <= e K sum_k |a|^(steps - 1 - k) |X_k|   (Frobenius)
with e = 2^-22, two binary digits below fp32's rounding for the sums.  bf16
results add their rounding, 2^-8 of the norm."""
import numpy as np
import pytest
import torch

import oracle
from cnn_cosmology_volumes_amd import cf
from gpu_util import host64, to_dev

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
NS = (5, 3.4445, -4.7750, 2.0315, 1e-7)
U = 2.0 ** -24


def bound(x, ns):
    steps, a, b, c, eps = ns
    k = abs(a) + 2 * abs(b) + 4 * abs(c)
    return 2.0 ** -22 * k * sum(abs(a) ** (steps - 1 - i) * np.linalg.norm(oracle.newton_schulz(x, i, a, b, c, eps))
                                for i in range(steps))


def gradient(rng, rows, cols, dtype=F32):
    r = min(4, rows, cols)
    g = rng.standard_normal((rows, r)) * 0.6 ** np.arange(r) @ rng.standard_normal((r, cols))
    g = (1e-3 * (g + rng.standard_normal((rows, cols)))).astype(np.float32)
    return host64(torch.from_numpy(g).to(dtype)).astype(np.float32)


def check_ns(got, x, ns=NS, dtype=F32):
    want = oracle.newton_schulz(x, *ns)
    tol = bound(x, ns) + (2.0 ** -8 * np.linalg.norm(want) if dtype == BF else 0.0)
    err = np.linalg.norm(host64(got) - want)
    assert err <= tol, (x.shape, err, tol)


SHAPES = [(1, 1), (1, 7), (7, 1), (1, 5000), (3, 5), (16, 16), (17, 63), (64, 64), (64, 65), (108, 32), (32, 108),
          (33, 1000), (101, 333), (130, 130), (300, 257), (1000, 300), (2111, 60), (515, 520), (700, 640), (1025, 1100)]


@pytest.mark.parametrize("dtype", [F32, BF], ids=["f32", "bf16"])
@pytest.mark.parametrize("shape", SHAPES, ids=["%dx%d" % s for s in SHAPES])
def test_newton_schulz(shape, dtype):
    x = gradient(np.random.default_rng(sum(shape)), *shape, dtype=dtype)
    xd = to_dev(x, dtype)
    keep = xd.clone()
    out = cf.cf_newton_schulz(cf.newton_schulz_params(), [xd])[0]
    assert out.dtype == dtype and torch.equal(xd, keep)
    check_ns(out, x, dtype=dtype)


@pytest.mark.parametrize("ns", [(1,) + NS[1:], (2,) + NS[1:], (3,) + NS[1:], (8, 1.5, -0.5, 0.0, 1e-7),
                                (5, 3.4445, -4.7750, 2.0315, 0.5)])
@pytest.mark.parametrize("shape", [(40, 50), (600, 530)])
def test_steps_and_coefficients(shape, ns):
    x = gradient(np.random.default_rng(4), *shape)
    out = cf.cf_newton_schulz(cf.newton_schulz_params(*ns), [to_dev(x, F32)])[0]
    check_ns(out, x, ns)


@pytest.mark.parametrize("scale", [1e-20, 1e-9, 1e12, 1e30])
@pytest.mark.parametrize("shape", [(24, 90), (530, 560)])
def test_gradients_of_any_size(shape, scale):
    x = gradient(np.random.default_rng(8), *shape) * np.float32(scale)
    out = cf.cf_newton_schulz(cf.newton_schulz_params(eps=1e-30), [to_dev(x, F32)])[0]
    check_ns(out, x, NS[:4] + (1e-30,))


@pytest.mark.parametrize("shape", [(5, 9), (70, 64), (600, 520)])
def test_zero_and_low_rank(shape):
    ns = cf.newton_schulz_params()
    zero = torch.zeros(shape, device="cuda")
    assert torch.equal(cf.cf_newton_schulz(ns, [zero])[0], zero)
    rng = np.random.default_rng(2)
    x = np.outer(rng.standard_normal(shape[0]), rng.standard_normal(shape[1])).astype(np.float32)
    x[:, ::3] = 0
    check_ns(cf.cf_newton_schulz(ns, [to_dev(x, F32)])[0], x)


def test_a_list_and_a_bad_matrix_in_it():
    """Matrices of a list do not touch each other, whatever their sizes; one
    with a NaN or an infinity is NaN itself and leaves the others alone."""
    rng = np.random.default_rng(12)
    shapes = [(108, 32), (3, 4), (900, 64), (520, 600), (1, 1), (16, 2000), (257, 256), (64, 3)]
    xs = [gradient(rng, *s) for s in shapes]
    xd = [to_dev(x, F32) for x in xs]
    ns = cf.newton_schulz_params()
    good = cf.cf_newton_schulz(ns, xd)
    for o, x in zip(good, xs):
        check_ns(o, x)
    for at, bad in ((0, float("nan")), (3, float("inf"))):
        bads = [x.clone() for x in xd]
        bads[at][1, 1] = bad
        out = cf.cf_newton_schulz(ns, bads)
        for i in range(len(xs)):
            if i == at:
                assert torch.isnan(out[i][1, 1])
            else:
                assert torch.equal(out[i], good[i]), (at, i)


def test_conv_weights_are_matrices():
    x = gradient(np.random.default_rng(3), 27 * 4, 32)
    ns = cf.newton_schulz_params()
    a = cf.cf_newton_schulz(ns, [to_dev(x, F32)])[0]
    b = cf.cf_newton_schulz(ns, [to_dev(x, F32).reshape(3, 3, 3, 4, 32)])[0]
    assert b.shape == (3, 3, 3, 4, 32) and torch.equal(a, b.reshape(108, 32))


LISTS = [[(108, 32), (864, 64), (64, 3)], [(300, 280), (1, 9), (2100, 96)], [(1200, 530)], [(7, 1)]]


@pytest.mark.parametrize("nesterov,scale,wd", [(True, "aspect", 0.01), (False, "rms", 0.0)])
@pytest.mark.parametrize("shapes", LISTS, ids=["-".join("%dx%d" % s for s in l) for l in LISTS])
def test_muon_steps(shapes, nesterov, scale, wd):
    rng = np.random.default_rng(len(shapes))
    f = lambda v: float(np.float32(v))
    lr, mu = f(0.02), f(0.95)
    hp = cf.muon_params(lr, momentum=mu, nesterov=nesterov, weight_decay=wd,
                        scale=cf.CF_MUON_SCALE_ASPECT if scale == "aspect" else cf.CF_MUON_SCALE_RMS)
    w = [to_dev(rng.standard_normal(s) * 0.1, F32) for s in shapes]
    m = [torch.zeros_like(t) for t in w]
    for step in range(3):
        gs = [gradient(rng, *s) for s in shapes]
        w0, m0 = [host64(t) for t in w], [host64(t) for t in m]
        cf.cf_muon(hp, w, [to_dev(g, F32) for g in gs], m)
        for i, s in enumerate(shapes):
            wo, mo = oracle.muon_step(w0[i], gs[i], m0[i], lr, mu, nesterov, f(wd), scale, NS)
            # two roundings of the momentum; the direction's own two, u of its norm, enter as u K a^4 / |u| would:
            # inside the bound's e
            assert np.all(np.abs(host64(m[i]) - mo) <= 2 * U * (np.abs(mu * m0[i]) + np.abs(gs[i])) + 1e-40)
            u = gs[i] + mu * mo if nesterov else mo
            fac = np.sqrt(max(1.0, s[1] / s[0])) if scale == "aspect" else 0.2 * np.sqrt(max(s))
            tol = lr * fac * bound(u, NS) + 3 * U * (np.linalg.norm(w0[i]) + np.linalg.norm(wo - w0[i]))
            assert np.linalg.norm(host64(w[i]) - wo) <= tol, (step, s)


def _list():
    rng = np.random.default_rng(21)
    shapes = [(108, 32), (530, 600), (2048, 128), (64, 3)]
    return [to_dev(gradient(rng, *s), F32) for s in shapes], rng


def test_reproducible_and_own_stream():
    xs, _ = _list()
    ns = cf.newton_schulz_params()
    a = cf.cf_newton_schulz(ns, xs)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    b = cf.cf_newton_schulz(ns, xs, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    for p, q in zip(a, b):
        assert torch.equal(p, q)


def test_graph_replays_equal_eager():
    gs, rng = _list()
    hp = cf.muon_params(0.02, weight_decay=0.01)
    we = [to_dev(rng.standard_normal(tuple(g.shape)) * 0.1, F32) for g in gs]
    wg = [t.clone() for t in we]
    me, mg = [torch.zeros_like(t) for t in we], [torch.zeros_like(t) for t in we]
    cf.cf_muon(hp, we, gs, me)
    cf.cf_muon(hp, wg, gs, mg)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        cf.cf_muon(hp, wg, gs, mg)
    for r in range(4):
        for t in gs:
            t.mul_(0.9)
        g.replay()
        cf.cf_muon(hp, we, gs, me)
        torch.cuda.synchronize()
        for p, q in zip(we + me, wg + mg):
            assert torch.equal(p, q), r
