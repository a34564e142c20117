"""GPU parity of linear layers (cf_linear_fwd / _bwd) against the fp64 oracle.

Tolerances, elementwise, from the roundings of the formulas (u = 2^-24):
  sums  of K products: (K + 2) u of the sum of the terms' magnitudes, whatever
        the order; bf16 products are exact in fp32
  pre   the sum's, plus u (|pre| + |bias|)
  y     |act'| <= 1.1 times pre's, plus the SiLU's own: exp's argument (u |z|),
        exp, reciprocal and two products, u (8 + 2 |z|) |act|, and u |y| of the
        residual's addition
  D     SiLU: u (16 + 4 |z|) (1 + |z|) |dy|; leaky ReLU: one product, u |dy|;
        for bf16 dX takes D rounded, 2^-8 |D|, dW takes D in two parts, 2^-16 |D|
  db    the terms' errors added, (rows + 2) u of the sum of magnitudes
bf16 outputs add 2^-8 of the value (half of the type's step)."""
import numpy as np
import pytest
import torch

import oracle
import synthdata as sd
from cnn_cosmology_volumes_amd import cf
from gpu_util import host64, to_dev

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
U = 2.0 ** -24
ACT = {"lrelu": cf.CF_ACT_LRELU, "silu": cf.CF_ACT_SILU}
TINY = 1e-37

SIZES = [
    (1, 33, 17), (3, 4096, 5), (4, 515, 300), (7, 1000, 1001), (8, 64, 4096), (13, 333, 129), (16, 2048, 512), (16, 40, 9000),
    (1, 1, 1), (1, 2048, 2048), (1, 16384, 128), (2, 3, 5), (8, 2048, 256), (16, 64, 3), (17, 129, 33),
    (5, 1, 70), (70, 7, 1), (63, 64, 65), (64, 64, 64), (65, 63, 127), (128, 128, 128), (129, 130, 131),
    (200, 8, 1024), (1000, 333, 1001), (1001, 1000, 8), (2048, 72, 40), (4099, 96, 96), (33000, 16, 24),
    (300, 2050, 260), (4096, 512, 512), (40000, 5, 3), (700, 1024, 1032),
]
IDS = ["x".join(map(str, s)) for s in SIZES]


def problem(rows, fin, fout, dtype, seed=0):
    rng = np.random.default_rng(rows * 7 + fin * 3 + fout + seed)
    bf = dtype == BF
    rnd = (lambda a: sd.bf16_round_f32(a.astype(np.float32))) if bf else (lambda a: a.astype(np.float32))
    x, w = rnd(rng.standard_normal((rows, fin)) + 0.25), rnd(rng.standard_normal((fin, fout)) / np.sqrt(fin))
    b = rng.standard_normal(fout).astype(np.float32)
    r, dy = rnd(rng.standard_normal((rows, fout))), rnd(rng.standard_normal((rows, fout)))
    return x, w, b, r, dy


def within(got, want, tol, dtype):
    got, want = host64(got), np.asarray(want)
    if dtype == BF:
        tol = tol + 2.0 ** -8 * (np.abs(want) + tol)
    worst = np.max(np.abs(got - want) / (tol + TINY))
    assert worst <= 1.0, worst


def check_fwd(pre, y, x, w, b, r, act, slope, dtype):
    po, yo = oracle.linear_fwd(x, w, b, act, slope, r)
    K = x.shape[1]
    mag = np.abs(x.astype(np.float64)) @ np.abs(w.astype(np.float64))
    ep = (K + 2) * U * mag + U * np.abs(po)
    if b is not None:
        ep = ep + U * np.abs(b)
    if pre is not None:
        within(pre, po, ep, dtype)
    a = yo - (0 if r is None else r)
    # (the second U: the sum that the residual is added to)
    within(y, yo, 1.1 * max(1.0, slope) * ep + U * (8 + 2 * np.abs(po)) * np.abs(a) + U * np.abs(yo), dtype)


def check_bwd(got, x, w, pre, dy, act, slope, dtype):
    dX, dW, db = got
    dxo, dwo, dbo = oracle.linear_bwd(x, w, pre, dy, act, slope)
    z, d = pre.astype(np.float64), np.abs(dy.astype(np.float64))
    D = np.abs(dy * oracle._act(z, act, slope)[1])
    plain = act == "lrelu" and slope == 1.0
    e = np.zeros_like(D) if plain else U * (16 + 4 * np.abs(z)) * (1 + np.abs(z)) * d if act == "silu" else U * D
    split = dtype == BF and not plain
    rows, fout = dy.shape
    ax, aw = np.abs(x.astype(np.float64)), np.abs(w.astype(np.float64))
    if dX is not None:
        within(dX, dxo, (e + (2.0 ** -8 * (D + e) if split else 0)) @ aw.T + (fout + 2) * U * (D @ aw.T) * 1.01, dtype)
    # a split D's two products, each rounded as a sum of that many terms
    within(dW, dwo, ax.T @ (e + (2.0 ** -16 * (D + e) if split else 0)) + (2 * rows + 2) * U * (ax.T @ D) * 1.01, F32)
    if db is not None:
        within(db, dbo, e.sum(axis=0) + (rows + 2) * U * D.sum(axis=0), F32)


def both(rows, fin, fout, dtype, act, slope, bias=True, residual=True, seed=0):
    x, w, b, r, dy = problem(rows, fin, fout, dtype, seed)
    xd, wd, dyd = to_dev(x, dtype), to_dev(w, dtype), to_dev(dy, dtype)
    bd, rd = to_dev(b, F32) if bias else None, to_dev(r, dtype) if residual else None
    pre, y = cf.cf_linear_fwd(xd, wd, bd, ACT[act], slope, R=rd)
    check_fwd(pre, y, x, w, b if bias else None, r if residual else None, act, slope, dtype)
    # the backward's definition starts from the pre that it is given
    check_bwd(cf.cf_linear_bwd(xd, wd, pre, dyd, ACT[act], slope), x, w, host64(pre), dy, act, slope, dtype)


@pytest.mark.parametrize("act,slope", [("lrelu", 0.3), ("silu", 0.0)])
@pytest.mark.parametrize("dtype", [F32, BF], ids=["f32", "bf16"])
@pytest.mark.parametrize("rows,fin,fout", SIZES, ids=IDS)
def test_matches_oracle(rows, fin, fout, dtype, act, slope):
    both(rows, fin, fout, dtype, act, slope)


@pytest.mark.parametrize("dtype", [F32, BF], ids=["f32", "bf16"])
@pytest.mark.parametrize("rows,fin,fout", [(1, 70, 30), (9, 512, 64), (300, 128, 96), (2000, 33, 61), (5000, 256, 256)])
def test_without_activation_bias_or_residual(rows, fin, fout, dtype):
    both(rows, fin, fout, dtype, "lrelu", 1.0, bias=False, residual=False)
    both(rows, fin, fout, dtype, "lrelu", 1.0, bias=True, residual=True, seed=1)
    both(rows, fin, fout, dtype, "lrelu", 0.0, bias=True, residual=False, seed=2)
    both(rows, fin, fout, dtype, "lrelu", 2.5, bias=False, residual=True, seed=3)


@pytest.mark.parametrize("dtype", [F32, BF], ids=["f32", "bf16"])
@pytest.mark.parametrize("rows,fin,fout", [(1, 2048, 2048), (3, 65, 33), (500, 96, 200)])
def test_optional_arguments(rows, fin, fout, dtype):
    x, w, b, r, dy = problem(rows, fin, fout, dtype)
    xd, wd, bd, dyd = to_dev(x, dtype), to_dev(w, dtype), to_dev(b, F32), to_dev(dy, dtype)
    pre, y = cf.cf_linear_fwd(xd, wd, bd, ACT["silu"])
    none, y2 = cf.cf_linear_fwd(xd, wd, bd, ACT["silu"], need_pre=False)
    assert none is None and torch.equal(y, y2)
    dx, dw, db = cf.cf_linear_bwd(xd, wd, pre, dyd, ACT["silu"])
    skipped, dw2, db2 = cf.cf_linear_bwd(xd, wd, pre, dyd, ACT["silu"], need_dx=False)
    assert skipped is None and torch.equal(dw, dw2) and torch.equal(db, db2)
    # outputs and workspace that the caller gives; pre is not needed without an activation
    out = [torch.full_like(xd, 7.0), torch.full((fin, fout), 7.0, device="cuda"), torch.full((fout,), 7.0, device="cuda")]
    ws = torch.empty(cf.cf_linear_workspace_size(cf.dtype_code(dtype), rows, fin, fout, True) + 256, dtype=torch.uint8,
                     device="cuda").fill_(255)
    got = cf.cf_linear_bwd(xd, wd, None, dyd, dX=out[0], dW=out[1], db=out[2], ws=ws)
    assert all(a is b for a, b in zip(got, out))
    check_bwd(got, x, w, host64(pre), dy, "lrelu", 1.0, dtype)


def test_voxels():
    """An NDHWC tensor: a 1^3 convolution."""
    x, w, b, r, _ = problem(2 * 3 * 4 * 5, 24, 40, BF)
    shape = (2, 3, 4, 5)
    pre, y = cf.cf_linear_fwd(to_dev(x, BF).reshape(*shape, 24), to_dev(w, BF), to_dev(b, F32), ACT["silu"],
                              R=to_dev(r, BF).reshape(*shape, 40))
    assert y.shape == pre.shape == (*shape, 40)
    check_fwd(pre.reshape(-1, 40), y.reshape(-1, 40), x, w, b, r, "silu", 0.0, BF)
    dx, dw, db = cf.cf_linear_bwd(to_dev(x, BF).reshape(*shape, 24), to_dev(w, BF), pre, y)
    assert dx.shape == (*shape, 24) and dw.shape == w.shape and db.shape == (40,)


@pytest.mark.parametrize("dtype", [F32, BF], ids=["f32", "bf16"])
@pytest.mark.parametrize("rows,fin,fout", [(3, 40, 24), (130, 72, 136), (130, 71, 135), (600, 512, 520)])
def test_what_is_not_finite_stays_in_its_row(rows, fin, fout, dtype):
    """Infinities and NaN reach the values whose formulas hold them, and no
    others (tiles and vectors that pass the end of a row read zeros)."""
    x, w, b, r, dy = problem(rows, fin, fout, dtype)
    x[rows // 2, fin - 1] = np.nan
    x[1, 0] = np.inf
    want = oracle.linear_fwd(x, w, b, "lrelu", 0.3, r)[1]
    _, y = cf.cf_linear_fwd(to_dev(x, dtype), to_dev(w, dtype), to_dev(b, F32), ACT["lrelu"], 0.3, R=to_dev(r, dtype))
    y = host64(y)
    assert np.array_equal(np.isnan(y), np.isnan(want)) and np.array_equal(np.isinf(y), np.isinf(want))
    clean = np.ones(rows, bool)
    clean[[1, rows // 2]] = False
    x[~clean] = 0
    check_fwd(None, torch.from_numpy(y[clean]), x[clean], w, b, r[clean], "lrelu", 0.3, dtype)
    # backward: a row of dY that is not finite leaves the other rows of dX alone
    x, w, b, r, dy = problem(rows, fin, fout, dtype)
    pre = oracle.linear_fwd(x, w, b, "silu", 0.0)[0].astype(np.float32)
    pred = to_dev(pre, dtype)
    d2 = dy.copy()
    d2[1, fout - 1] = np.inf
    a = host64(cf.cf_linear_bwd(to_dev(x, dtype), to_dev(w, dtype), pred, to_dev(dy, dtype), ACT["silu"])[0])
    dx, dw, db = (host64(v) for v in cf.cf_linear_bwd(to_dev(x, dtype), to_dev(w, dtype), pred, to_dev(d2, dtype),
                                                      ACT["silu"]))
    assert not np.isfinite(dx[1]).any()
    assert np.array_equal(np.delete(a, 1, 0), np.delete(dx, 1, 0))
    assert np.isinf(db[-1]) and np.isfinite(db[:-1]).all()
    assert np.isinf(dw[:, -1]).all() and np.isfinite(dw[:, :-1]).all()


@pytest.mark.parametrize("dtype", [F32, BF], ids=["f32", "bf16"])
def test_rows_behind_the_last_stay(dtype):
    """Outputs are written to their last value and no further."""
    rows, fin, fout = 37, 45, 51
    x, w, b, r, dy = problem(rows, fin, fout, dtype)
    room = lambda n, t: torch.full((n + 4096,), 3.0, dtype=t, device="cuda")  # noqa: E731
    keep = [(room(rows * fout, dtype), rows * fout), (room(rows * fout, dtype), rows * fout),
            (room(rows * fin, dtype), rows * fin), (room(fin * fout, F32), fin * fout), (room(fout, F32), fout)]
    v = [t[:n] for t, n in keep]
    xd, wd, dyd = to_dev(x, dtype), to_dev(w, dtype), to_dev(dy, dtype)
    pre, y = cf.cf_linear_fwd(xd, wd, to_dev(b, F32), ACT["silu"], pre=v[0].view(rows, fout), Y=v[1].view(rows, fout))
    got = cf.cf_linear_bwd(xd, wd, pre, dyd, ACT["silu"], dX=v[2].view(rows, fin), dW=v[3].view(fin, fout), db=v[4])
    check_fwd(pre, y, x, w, b, None, "silu", 0.0, dtype)
    check_bwd(got, x, w, host64(pre), dy, "silu", 0.0, dtype)
    for t, n in keep:
        assert bool((t[n:] == 3.0).all())


@pytest.mark.parametrize("dtype", [F32, BF], ids=["f32", "bf16"])
@pytest.mark.parametrize("rows,fin,fout", [(2, 4096, 64), (5000, 65, 31), (20000, 64, 64)])
def test_reproducible(rows, fin, fout, dtype):
    x, w, b, r, dy = problem(rows, fin, fout, dtype)
    xd, wd, bd, dyd = to_dev(x, dtype), to_dev(w, dtype), to_dev(b, F32), to_dev(dy, dtype)
    first = None
    for _ in range(3):
        pre, y = cf.cf_linear_fwd(xd, wd, bd, ACT["silu"])
        got = (pre, y, *cf.cf_linear_bwd(xd, wd, pre, dyd, ACT["silu"]))
        first = first or got
        assert all(torch.equal(a, b) for a, b in zip(got, first))


def test_gradient_against_differences():
    """The gradients as the derivative of the library's own forward: central
    differences in fp32 along random directions, step h = 2^-5 of the inputs."""
    rows, fin, fout, h = 50, 30, 20, 2.0 ** -5
    x, w, b, r, dy = (to_dev(v, F32) for v in problem(rows, fin, fout, F32))
    f = lambda x, w, b: (cf.cf_linear_fwd(x, w, b, ACT["silu"], R=r)[1].double() * dy.double()).sum().item()  # noqa: E731
    pre, _ = cf.cf_linear_fwd(x, w, b, ACT["silu"])
    grads = cf.cf_linear_bwd(x, w, pre, dy, ACT["silu"])
    gen = torch.Generator(device="cuda").manual_seed(1)
    for k, (a, g) in enumerate(zip((x, w, b), grads)):
        e = torch.randn(a.shape, generator=gen, device="cuda")
        e = e / e.norm()
        at = lambda s: f(*[t + s * e if j == k else t for j, t in enumerate((x, w, b))])  # noqa: E731
        slope = (at(h) - at(-h)) / (2 * h)
        # truncation h^2 / 6 |f'''|, |silu'''| <= 1 and sum |dy| |dpre|^3 <= max|dy| max|x or w|^3 sqrt(n)^3-like terms
        # stay below 50 here; rounding u sum |y dy| / h
        noise = U * float((cf.cf_linear_fwd(x, w, b, ACT["silu"], R=r)[1].double() * dy.double()).abs().sum()) / h
        assert abs(slope - float((g.double() * e.double()).sum())) <= h * h / 6 * 50 + 8 * noise


def test_past_2_31_elements():
    """64-bit offsets: rows behind 2^31 elements of X, pre, Y and their gradients."""
    fin, fout, rows = 8, 512, (1 << 22) + 513
    gen = torch.Generator(device="cuda").manual_seed(5)
    x = torch.randn(rows, fin, generator=gen, device="cuda").to(BF)
    w = torch.randn(fin, fout, generator=gen, device="cuda").to(BF)
    pre, y = cf.cf_linear_fwd(x, w, None, ACT["silu"])
    dx, dw, db = cf.cf_linear_bwd(x, w, pre, y, ACT["silu"])
    at = slice(rows - 700, rows)
    xs, ws = host64(x[at]), host64(w)
    check_fwd(pre[at], y[at], xs, ws, None, None, "silu", 0.0, BF)
    part = cf.cf_linear_bwd(x[at].clone(), w, pre[at].clone(), y[at].clone(), ACT["silu"])[0]
    assert torch.equal(part, dx[at])
    total = torch.zeros(fout, dtype=torch.float64, device="cuda")
    for i in range(0, rows, 1 << 20):
        p, d = pre[i:i + (1 << 20)].double(), y[i:i + (1 << 20)].double()
        s = torch.sigmoid(p)
        total += (d * s * (1 + p * (1 - s))).sum(0)
    assert float((db.double() - total).abs().max() / total.abs().max()) < 1e-5


@pytest.mark.parametrize("dtype", [F32, BF], ids=["f32", "bf16"])
@pytest.mark.parametrize("rows,fin,fout", [(16700, 264, 776), (33001, 136, 520), (16640, 512, 256), (9000, 1000, 1001)])
def test_large_tiles(rows, fin, fout, dtype):
    """Sizes that take the largest tiles, whole ones and ones that the result cuts."""
    both(rows, fin, fout, dtype, "silu", 0.0)
    both(rows, fin, fout, dtype, "lrelu", 1.0, bias=False, residual=False, seed=1)


@pytest.mark.parametrize("dtype", [F32, BF], ids=["f32", "bf16"])
@pytest.mark.parametrize("rows,fin,fout", [(70000, 2, 1), (45001, 13, 13), (60000, 254, 16), (20001, 64, 9)])
def test_narrow(rows, fin, fout, dtype):
    """Long reductions to few results: hundreds of splits, joined by many threads a result."""
    both(rows, fin, fout, dtype, "silu", 0.0)
    both(rows, fin, fout, dtype, "lrelu", 1.0, residual=False, seed=1)
