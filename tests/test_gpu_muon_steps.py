"""Newton-Schulz and Muon with many steps, on every path: one block with the
whole matrix, shorter sides up to 64, fp64 rounds with tiles of 16 and of 32,
and split fp16 products.

With f(s) = a s + b s^3 + c s^5 a step maps each singular value s to f(s), and
an error E of X to one of at most g |E|, g the largest of |f'(s)| and |f(s)/s|
over the range of X's singular values.  A step computed with products of
relative error 2^-22 adds 2^-22 K |X_k|, K = |a| + 2 |b| + 4 |c|, so
  |out - exact| <= 2^-22 K sum_k |X_k| g_{k+1} ... g_{steps-1}     (Frobenius)
and bf16 results add 2^-8 |out|.  Each check first asserts that this is below
a hundredth of the result: a tolerance that says nothing would pass anything."""
import functools

import numpy as np
import pytest
import torch

from cnn_cosmology_volumes_amd import cf
from gpu_util import host64, to_dev

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
MUON = (3.4445, -4.7750, 2.0315)
CONVERGENT = [(1.875, -1.25, 0.375), (2.0, -1.5, 0.5), (1.5, -0.5, 0.0)]      # f(1) = 1, f'(1) = 0
EPS = 1e-7

SHAPES = [(16, 40), (48, 128), (128, 48),      # one block
          (64, 700), (3000, 60),               # U U^T, one block, s Q U
          (128, 2048), (319, 200),             # rounds, tiles of 16
          (449, 4300),                         # rounds, tiles of 32
          (530, 600)]                          # split products
IDS = ["%dx%d" % s for s in SHAPES]


def wide(x):
    return x if x.shape[0] <= x.shape[1] else x.T


def spectrum(x):
    """Eigenvalues and vectors of X X^T on the shorter side, in float64."""
    t = wide(np.asarray(x, np.float64))
    w, v = np.linalg.eigh(t @ t.T)
    return np.maximum(w, 0.0), v


@functools.lru_cache(maxsize=None)
def full_rank(shape, dtype=F32, seed=0):
    """A matrix with singular values within a factor of ten of each other, and
    the singular values of X_0."""
    rng, m, n = np.random.default_rng(sum(shape) + seed), min(shape), max(shape)
    q = np.linalg.qr(rng.standard_normal((n, m)))[0]
    p = np.linalg.qr(rng.standard_normal((m, m)))[0]
    x = ((q * rng.uniform(0.1, 1.0, m)) @ p).astype(np.float32)
    x = np.ascontiguousarray(x if shape[0] > shape[1] else x.T)
    x = host64(torch.from_numpy(x).to(dtype)).astype(np.float32)
    s = np.sqrt(spectrum(x)[0])
    return x, s / (np.sqrt(np.sum(s * s)) + EPS)


def low_rank(rng, rows, cols, r=4):
    return (rng.standard_normal((rows, r)) @ rng.standard_normal((r, cols))).astype(np.float32)


def tolerance(s, steps, coef):
    a, b, c = coef
    k, total = abs(a) + 2 * abs(b) + 4 * abs(c), 0.0
    for _ in range(steps):
        t = np.linspace(s.min(), s.max(), 2001)
        g = max(np.abs(a + 3 * b * t ** 2 + 5 * c * t ** 4).max(), np.abs(a + b * t ** 2 + c * t ** 4).max())
        total = total * g + 2.0 ** -22 * k * np.linalg.norm(s)
        s = np.abs(a * s + b * s ** 3 + c * s ** 5)
    return total


def definition(x, steps, coef):
    t = torch.from_numpy(np.ascontiguousarray(wide(x))).cuda().double()
    t = t / (t.norm() + EPS)
    for _ in range(steps):
        g = t @ t.t().contiguous()
        t = coef[0] * t + (coef[1] * g + coef[2] * (g @ g)) @ t
    t = t.cpu().numpy()
    return t if x.shape[0] <= x.shape[1] else t.T


def call(x, steps, coef, dtype=F32):
    return cf.cf_newton_schulz(cf.newton_schulz_params(steps, *coef, eps=EPS), [to_dev(x, dtype)])[0]


@pytest.mark.parametrize("dtype", [F32, BF], ids=["f32", "bf16"])
@pytest.mark.parametrize("steps,coef", [(9, MUON), (10, MUON), (16, CONVERGENT[0]), (32, CONVERGENT[0]),
                                        (20, CONVERGENT[1]), (30, CONVERGENT[2])])
@pytest.mark.parametrize("shape", SHAPES, ids=IDS)
def test_full_rank(shape, steps, coef, dtype):
    x, s = full_rank(shape, dtype)
    want, tol = definition(x, steps, coef), tolerance(s, steps, coef)
    assert tol < 0.01 * np.linalg.norm(want)
    if dtype == BF:
        tol += 2.0 ** -8 * np.linalg.norm(want)
    err = np.linalg.norm(host64(call(x, steps, coef, dtype)) - want)
    assert err <= tol, (err, tol)


@pytest.mark.parametrize("shape", SHAPES, ids=IDS)
def test_convergent_steps_give_the_polar_factor(shape):
    """32 steps end at (X X^T)^(-1/2) X, whatever the path to it."""
    x, s = full_rank(shape)
    w, v = spectrum(x)
    polar = (v / np.sqrt(w)) @ v.T @ wide(x).astype(np.float64)
    tol = tolerance(s, 32, CONVERGENT[0])
    assert tol < 0.01 * np.sqrt(len(s))
    out = wide(host64(call(x, 32, CONVERGENT[0])))
    assert np.linalg.norm(out - polar) <= tol
    assert np.linalg.norm(out @ out.T - np.eye(len(s))) <= 2 * tol + tol * tol


def largest_value(coef):
    """Of f over the singular values that occur: [0, 1], then f's own range."""
    top = 1.0
    for _ in range(3):
        t = np.linspace(0.0, top, 100001)
        big = np.abs(coef[0] * t + coef[1] * t ** 3 + coef[2] * t ** 5).max()
        top = max(top, big)
    return big


@pytest.mark.parametrize("steps,coef", [(16, MUON), (20, MUON), (32, MUON), (32, CONVERGENT[0]), (32, CONVERGENT[1])])
@pytest.mark.parametrize("shape", SHAPES, ids=IDS)
def test_rank_deficient_stays_bounded(shape, steps, coef):
    """Directions that U lacks hold rounding errors, which so many steps raise
    to singular values near 1 in any finite precision; f's range bounds them.
    On top comes the error of the last product of a factor of norm 2^14.5 at
    most with X, three roundings of 2^-24 of its terms: 3 2^-9.5 |X|."""
    x = low_rank(np.random.default_rng(5), *shape)
    out = wide(host64(call(x, steps, coef)))
    assert np.isfinite(out).all()
    err = 3 * 2.0 ** -9.5 * np.sqrt(min(shape))
    assert np.sqrt(np.linalg.eigvalsh(out @ out.T).max()) <= largest_value(coef) * (1 + err)
    if coef == MUON:
        return
    # the directions that U has come out as f takes them: a quarter of that error is already a part of all others
    t = wide(x).astype(np.float64)
    w, v = spectrum(x)
    w, v = w[-4:], v[:, -4:]
    s = np.sqrt(w) / np.sqrt(w.sum())
    for _ in range(steps):
        s = coef[0] * s + coef[1] * s ** 3 + coef[2] * s ** 5
    core = v.T @ out @ (t.T @ v / np.sqrt(w))
    assert np.linalg.norm(core - np.diag(s)) <= 0.25 * err


@pytest.mark.parametrize("shape", [(16, 40), (64, 700), (128, 2048), (530, 600)])
def test_zero_nan_and_infinity(shape):
    assert not call(np.zeros(shape, np.float32), 32, MUON).any()
    for bad in (np.nan, np.inf):
        x = full_rank(shape)[0].copy()
        x[3, 7] = bad
        assert torch.isnan(call(x, 20, MUON)[3, 7])


def test_lists_of_many_steps():
    shapes = [(108, 32), (300, 64), (1, 1), (64, 3), (1, 500), (530, 600), (257, 256)]
    xs = [full_rank(s, seed=7) for s in shapes]
    ns = cf.newton_schulz_params(32, *CONVERGENT[0])
    for (x, s), o in zip(xs, cf.cf_newton_schulz(ns, [to_dev(x, F32) for x, _ in xs])):
        want, tol = definition(x, 32, CONVERGENT[0]), tolerance(s, 32, CONVERGENT[0])
        assert tol < 0.01 * np.linalg.norm(want)
        assert np.linalg.norm(host64(o) - want) <= tol, x.shape


@pytest.mark.parametrize("nesterov", [False, True])
def test_muon_of_low_rank_gradients(nesterov):
    """A dense layer's gradient has the batch's rank at most; an update has
    singular values up to lr scale(rows, cols) max f = 1.21, and the errors of
    test_rank_deficient_stays_bounded, 10% here."""
    shapes = [(108, 32), (64, 700), (2048, 128), (600, 530)]
    rng = np.random.default_rng(8)
    hp = cf.muon_params(0.02, nesterov=nesterov, ns=cf.newton_schulz_params(20, *MUON))
    w = [to_dev(0.1 * rng.standard_normal(s), F32) for s in shapes]
    m = [torch.zeros_like(t) for t in w]
    for _ in range(3):
        before = [host64(t) for t in w]
        cf.cf_muon(hp, w, [to_dev(1e-3 * low_rank(rng, *s), F32) for s in shapes], m)
        for t, old, s in zip(w, before, shapes):
            d = wide(host64(t) - old)
            assert np.isfinite(d).all()
            assert np.sqrt(np.linalg.eigvalsh(d @ d.T).max()) <= 0.02 * np.sqrt(max(1.0, s[1] / s[0])) * 1.21 * 1.1, s


@pytest.mark.parametrize("dtype", [F32, BF], ids=["f32", "bf16"])
@pytest.mark.parametrize("shape", SHAPES, ids=IDS)
def test_nothing_is_read_from_the_workspace_and_replays(shape, dtype):
    ns = cf.newton_schulz_params(20, *CONVERGENT[0])
    xd = to_dev(full_rank(shape, dtype)[0], dtype)
    size = cf.lib().cf_newton_schulz_workspace_size(cf.dtype_code(dtype), 1, *cf._mat_sizes([xd]))
    got = []
    for fill in (0xFF, 0x7B):
        ws = torch.full((size,), fill, dtype=torch.uint8, device="cuda")
        got.append(cf.cf_newton_schulz(ns, [xd], ws=ws)[0])
    assert torch.isfinite(got[0].float()).all() and torch.equal(got[0], got[1])
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = cf.cf_newton_schulz(ns, [xd])[0]
    for _ in range(3):
        xd.copy_(xd.flip(0).contiguous() * 0.5)
        want = cf.cf_newton_schulz(ns, [xd])[0]
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(held, want)
