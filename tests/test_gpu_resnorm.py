"""GPU parity of the residual join with its norms (cf_resnorm_fwd / _bwd)
against the fp64 oracle.

Tolerances, elementwise, from the roundings of the formulas (u = 2^-24).  A sum
over a row goes through at most 16 additions in a lane and 8 between lanes, so
it is off by at most g = 32 u of the sum of its terms' magnitudes (with the
terms' own roundings):
  hat   a normalised value: the centring's and the statistics' errors,
        2 g (|hat| + mean |hat|)
  join  r: |gate gpost| hat's, and 6u of the magnitudes of its terms
  y     r's error through the norm, rstd (er + mean er) + |hat| rstd mean(er |hat|),
        plus hat's, times |gpre|, plus 3u of its terms
  through a norm: every factor's error as it stands in the formula
  column sums: a lane adds at most rows / 1024 + 8 terms in fp32, lanes and
        waves 8 more, blocks in fp64: u (rows / 1024 + 24) of the magnitudes
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
G = 32 * U
EPS = 1e-5
KIND = {"rms": cf.CF_NORM_RMS, "layer": cf.CF_NORM_LAYER}
TINY = 1e-37

SHAPES = [(1, 1, 1, 1, 1), (1, 1, 1, 1, 8), (1, 1, 1, 3, 2), (2, 3, 1, 2, 7), (3, 2, 2, 2, 16), (1, 4, 4, 4, 17),
          (2, 3, 5, 2, 31), (2, 4, 4, 4, 32), (2, 5, 3, 4, 60), (1, 8, 8, 8, 64), (4, 2, 3, 3, 100), (2, 4, 4, 5, 128),
          (3, 3, 3, 3, 200), (1, 4, 4, 4, 256), (2, 2, 3, 3, 333), (2, 3, 3, 2, 512), (2, 1, 3, 3, 777), (1, 3, 2, 2, 1024),
          (2, 2, 1, 3, 1500), (3, 1, 2, 2, 2048), (1, 2, 2, 3, 3001), (2, 1, 2, 2, 4096), (2, 16, 17, 19, 48),
          (9, 1, 1, 1, 40), (1500, 1, 1, 1, 24), (1100, 1, 2, 1, 300), (3, 20, 21, 22, 12)]
IDS = ["x".join(map(str, s)) for s in SHAPES]


def problem(shape, dtype, post=True, offset=True, gate_n=0, seed=0):
    rng = np.random.default_rng(sum(shape) + seed)
    c = shape[-1]
    rnd = (lambda a: sd.bf16_round_f32(a.astype(np.float32))) if dtype == BF else (lambda a: a.astype(np.float32))
    t = {n: rnd(rng.standard_normal(shape) * rng.uniform(0.5, 1.5, c) + 0.4) for n in ("x", "f", "r", "dr", "dy")}
    vec = lambda lo, hi: rng.uniform(lo, hi, c).astype(np.float32)  # noqa: E731
    p = {"gpre": vec(-1.5, 1.5)}
    if offset:
        p["bpre"] = vec(-0.5, 0.5)
    if post:
        p["gpost"] = vec(-1.5, 1.5)
        if offset:
            p["bpost"] = vec(-0.5, 0.5)
    if gate_n:
        p["gate"] = rng.uniform(-1, 1, (gate_n, c)).astype(np.float32)
    return t, p


def within(got, want, tol, dtype):
    got = host64(got)
    if dtype == BF:
        tol = tol + 2.0 ** -8 * (np.abs(want) + tol)
    worst = np.max(np.abs(got - want) / (tol + TINY))
    assert worst <= 1.0, worst


def mean(a):
    return a.mean(axis=-1, keepdims=True)


def hat_error(hat):
    return 2 * G * (np.abs(hat) + mean(np.abs(hat)))


def through(d, ed, hat, eh, rstd):
    """Error of a gradient d (off by ed) through the norm; rstd is off by g."""
    ad, ah = np.abs(d), np.abs(hat)
    c1, c0 = np.abs(mean(d * hat)), np.abs(mean(d))
    e1 = mean(ed * ah + ad * eh) + G * mean(ad * ah)
    return rstd * (ed + ah * e1 + eh * c1 + mean(ed) + G * mean(ad) + 2 * G * (ad + ah * c1 + c0))


def check_fwd(R, Y, t, p, kind, alpha, dtype, eps=EPS):
    shape = t["x"].shape
    c = shape[-1]
    ro, yo = oracle.resnorm_fwd(t["x"], t["f"], kind, eps, alpha=alpha, **p)
    gate = np.abs(oracle._per_sample(p.get("gate"), shape))
    h, eh = t["f"].astype(np.float64), 0.0
    po, bo = np.abs(oracle._vec(p.get("gpost"), c, 1.0)), np.abs(oracle._vec(p.get("bpost"), c, 0.0))
    if "gpost" in p:
        h, _ = oracle.row_norm(h, kind, eps)
        eh = hat_error(h)
    er = gate * po * eh + 6 * U * (gate * (po * np.abs(h) + bo) + np.abs(alpha * t["x"]))
    within(R, ro, er, dtype)
    if Y is None:
        return
    hat, rstd = oracle.row_norm(ro, kind, eps)
    ey = rstd * (er + mean(er)) + np.abs(hat) * rstd * mean(er * np.abs(hat)) + hat_error(hat)
    gp, bp = np.abs(oracle._vec(p.get("gpre"), c, 1.0)), np.abs(oracle._vec(p.get("bpre"), c, 0.0))
    within(Y, yo, gp * ey + 3 * U * (gp * np.abs(hat) + bp), dtype)


def check_bwd(got, t, p, kind, alpha, dtype, dr=True, dy=True, eps=EPS):
    dX, dF, dgpre, dbpre, dgpost, dbpost, dgate = got
    shape, lead = t["f"].shape, (0, 1, 2, 3)
    c, rows = shape[-1], int(np.prod(shape[:4]))
    want = oracle.resnorm_bwd(t["f"], t["r"], t["dr"] if dr else None, t["dy"] if dy else None, kind, eps, alpha=alpha, **p)
    S = U * (rows / 1024 + 24)
    d, ed = (t["dr"].astype(np.float64), 0.0) if dr else (np.zeros(shape), 0.0)
    if dy:
        hat, rstd = oracle.row_norm(t["r"], kind, eps)
        eh, ady = hat_error(hat), np.abs(t["dy"].astype(np.float64))
        if dgpre is not None:
            within(dgpre, want["dgpre"], (ady * eh).sum(axis=lead) + S * (ady * np.abs(hat)).sum(axis=lead), F32)
        if dbpre is not None:
            within(dbpre, want["dbpre"], S * ady.sum(axis=lead), F32)
        v = t["dy"] * oracle._vec(p.get("gpre"), c, 1.0)
        ed = through(v, U * np.abs(v), hat, eh, rstd)
        d = d + oracle.row_norm_bwd(v, hat, rstd, kind)
        ed = ed + 2 * U * np.abs(d)
    within(dX, want["dx"], np.abs(alpha) * ed + 2 * U * np.abs(want["dx"]), dtype)
    gate = oracle._per_sample(p.get("gate"), shape)
    h, eh, rstd = t["f"].astype(np.float64), 0.0, None
    if "gpost" in p:
        h, rstd = oracle.row_norm(h, kind, eps)
        eh = hat_error(h)
    ag, ad, ah = np.abs(gate), np.abs(d), np.abs(h)
    e_hat = ed * ah + ad * eh                       # of the terms d h
    if "gpost" in p:
        u = gate * p["gpost"] * d
        within(dF, want["df"], through(u, np.abs(gate * p["gpost"]) * ed + 3 * U * np.abs(u), h, eh, rstd), dtype)
        within(dgpost, want["dgpost"], (ag * e_hat).sum(axis=lead) + (S + 4 * U) * (ag * ad * ah).sum(axis=lead), F32)
        if dbpost is not None:
            within(dbpost, want["dbpost"], (ag * (ed + 0 * ad)).sum(axis=lead) + (S + 4 * U) * (ag * ad).sum(axis=lead), F32)
    else:
        within(dF, want["df"], ag * ed + 2 * U * np.abs(want["df"]), dtype)
    if dgate is not None:
        po, bo = np.abs(oracle._vec(p.get("gpost"), c, 1.0)), np.abs(oracle._vec(p.get("bpost"), c, 0.0))
        e = (po * e_hat + bo * (ed + 0 * ad)).sum(axis=(1, 2, 3)) + (S + 6 * U) * (po * ad * ah + bo * ad).sum(axis=(1, 2, 3))
        one = dgate.shape[0] == 1 and shape[0] > 1
        within(dgate, want["dgate"], e.sum(axis=0, keepdims=True) if one else e, F32)


def dev(p):
    return {k: to_dev(v, F32) for k, v in p.items()}


def run(shape, dtype, kind, post=True, offset=True, gate_n=0, alpha=1.0, seed=0):
    t, p = problem(shape, dtype, post, offset, gate_n, seed)
    g, q = {k: to_dev(v, dtype) for k, v in t.items()}, dev(p)
    R, Y = cf.cf_resnorm_fwd(g["x"], g["f"], KIND[kind], EPS, alpha=alpha, **q)
    check_fwd(R, Y, t, p, kind, alpha, dtype)
    got = cf.cf_resnorm_bwd(g["f"], g["r"], g["dr"], g["dy"], KIND[kind], EPS, alpha=alpha, **q)
    check_bwd(got, t, p, kind, alpha, dtype)
    return got


@pytest.mark.parametrize("kind", ["rms", "layer"])
@pytest.mark.parametrize("dtype", [F32, BF], ids=["f32", "bf16"])
@pytest.mark.parametrize("shape", SHAPES, ids=IDS)
def test_matches_oracle(shape, dtype, kind):
    run(shape, dtype, kind, gate_n=shape[0], alpha=0.8)


@pytest.mark.parametrize("post", [False, True])
@pytest.mark.parametrize("gate_n", [0, 1, 3])
@pytest.mark.parametrize("kind", ["rms", "layer"])
@pytest.mark.parametrize("shape", [(3, 2, 5, 3, 24), (3, 1, 2, 2, 45), (3, 1, 1, 3, 1300)])
def test_parts_of_the_operator(shape, kind, gate_n, post):
    for dtype in (F32, BF):
        run(shape, dtype, kind, post, True, gate_n, -1.25)
        run(shape, dtype, kind, post, False, gate_n, 1.0, seed=1)


@pytest.mark.parametrize("dtype", [F32, BF], ids=["f32", "bf16"])
@pytest.mark.parametrize("kind", ["rms", "layer"])
def test_optional_tensors(kind, dtype):
    shape = (2, 3, 3, 3, 72)
    t, p = problem(shape, dtype, gate_n=2)
    g, q = {k: to_dev(v, dtype) for k, v in t.items()}, dev(p)
    R, Y = cf.cf_resnorm_fwd(g["x"], g["f"], KIND[kind], EPS, need_y=False, **q)
    assert Y is None
    check_fwd(R, None, t, p, kind, 1.0, dtype)
    assert torch.equal(R, cf.cf_resnorm_fwd(g["x"], g["f"], KIND[kind], EPS, **q)[0])
    # the last block: no further norm
    got = cf.cf_resnorm_bwd(g["f"], None, g["dr"], None, KIND[kind], EPS, **q)
    assert got[2] is None and got[3] is None
    check_bwd(got, t, p, kind, 1.0, dtype, dy=False)
    got = cf.cf_resnorm_bwd(g["f"], g["r"], None, g["dy"], KIND[kind], EPS, **q)
    check_bwd(got, t, p, kind, 1.0, dtype, dr=False)
    # no vectors at all
    bare = {}
    R, Y = cf.cf_resnorm_fwd(g["x"], g["f"], KIND[kind], EPS)
    check_fwd(R, Y, t, bare, kind, 1.0, dtype)
    got = cf.cf_resnorm_bwd(g["f"], g["r"], g["dr"], g["dy"], KIND[kind], EPS)
    assert all(v is None for v in got[2:])
    check_bwd(got, t, bare, kind, 1.0, dtype)
    # a gate as a plain vector
    one = to_dev(p["gate"][0], F32)
    got = cf.cf_resnorm_bwd(g["f"], g["r"], g["dr"], g["dy"], KIND[kind], EPS, gate=one)
    assert got[6].shape == one.shape
    assert torch.equal(got[6], cf.cf_resnorm_bwd(g["f"], g["r"], g["dr"], g["dy"], KIND[kind], EPS, gate=one[None])[6][0])


@pytest.mark.parametrize("c", [24, 300, 2000])
def test_rows_without_spread(c):
    """Rows of zeros, and rows of one value: a layer norm of 0, no NaN."""
    shape = (1, 1, 1, 4, c)
    x, f = np.zeros(shape, np.float32), np.zeros(shape, np.float32)
    x[0, 0, 0, 1], f[0, 0, 0, 1] = 3.0, 1.0
    x[0, 0, 0, 2] = 1e4
    for kind in KIND:
        R, Y = cf.cf_resnorm_fwd(to_dev(x, F32), to_dev(f, F32), KIND[kind], EPS)
        ro, yo = oracle.resnorm_fwd(x, f, kind, EPS)
        assert np.array_equal(host64(R), ro)
        # constant rows: x - mean is exact in the end, up to the second mean's rounding
        assert np.all(np.abs(host64(Y) - yo) <= (G if kind == "rms" else 2.0 ** -20)), kind
        one = torch.ones(shape, device="cuda")
        got = cf.cf_resnorm_bwd(to_dev(f, F32), R, None, one, KIND[kind], EPS, gpost=torch.ones(c, device="cuda"))
        assert all(bool(torch.isfinite(v).all()) for v in got if v is not None)


def test_large_offsets():
    """Layer norm of rows whose mean is 3000 spreads: x - mean keeps the digits
    that x has."""
    rng = np.random.default_rng(4)
    shape = (1, 2, 3, 4, 500)
    x = (3000 + rng.standard_normal(shape)).astype(np.float32)
    f = np.zeros(shape, np.float32)
    R, Y = cf.cf_resnorm_fwd(to_dev(x, F32), to_dev(f, F32), KIND["layer"], EPS)
    assert np.array_equal(host64(R), x)
    hat = oracle.row_norm(x, "layer", EPS)[0]
    # x - m and m2 (each of the centred values' size), the statistics: no term grows with the mean
    assert np.all(np.abs(host64(Y) - hat) <= 2 * G * (np.abs(hat) + mean(np.abs(hat))))


@pytest.mark.parametrize("dtype", [F32, BF], ids=["f32", "bf16"])
@pytest.mark.parametrize("c", [12, 45, 1024, 2050])
def test_what_is_not_finite_stays_in_its_row(c, dtype):
    shape = (2, 1, 2, 3, c)
    t, p = problem(shape, dtype, gate_n=2)
    q = dev(p)
    for bad in (np.nan, np.inf):
        x = t["x"].copy()
        x[0, 0, 1, 1, c - 1] = bad
        a = cf.cf_resnorm_fwd(to_dev(t["x"], dtype), to_dev(t["f"], dtype), KIND["layer"], EPS, **q)
        b = cf.cf_resnorm_fwd(to_dev(x, dtype), to_dev(t["f"], dtype), KIND["layer"], EPS, **q)
        for u, v in zip(a, b):
            u, v = host64(u).reshape(-1, c), host64(v).reshape(-1, c)
            assert np.array_equal(np.delete(u, 4, 0), np.delete(v, 4, 0))
        assert not np.isfinite(host64(b[1]).reshape(-1, c)[4]).any()
        dy = t["dy"].copy()
        dy[0, 0, 1, 1, 0] = bad
        arg = [to_dev(t[k], dtype) for k in ("f", "r", "dr")]
        a = cf.cf_resnorm_bwd(*arg, to_dev(t["dy"], dtype), KIND["rms"], EPS, **q)
        b = cf.cf_resnorm_bwd(*arg, to_dev(dy, dtype), KIND["rms"], EPS, **q)
        for u, v in zip(a[:2], b[:2]):
            u, v = host64(u).reshape(-1, c), host64(v).reshape(-1, c)
            assert np.array_equal(np.delete(u, 4, 0), np.delete(v, 4, 0)) and not np.isfinite(v[4]).any()
        assert torch.equal(a[6][1], b[6][1])                # the other sample's gate


@pytest.mark.parametrize("dtype", [F32, BF], ids=["f32", "bf16"])
def test_rows_behind_the_last_stay(dtype):
    shape = (1, 1, 3, 7, 43)
    n = int(np.prod(shape))
    t, p = problem(shape, dtype, gate_n=1)
    g, q = {k: to_dev(v, dtype) for k, v in t.items()}, dev(p)
    room = [torch.full((n + 4096,), 3.0, dtype=dtype, device="cuda") for _ in range(4)]
    v = [r[:n].view(shape) for r in room]
    cf.cf_resnorm_fwd(g["x"], g["f"], KIND["layer"], EPS, R=v[0], Y=v[1], **q)
    check_fwd(v[0], v[1], t, p, "layer", 1.0, dtype)
    got = cf.cf_resnorm_bwd(g["f"], g["r"], g["dr"], g["dy"], KIND["layer"], EPS, dX=v[2], dF=v[3], **q)
    check_bwd(got, t, p, "layer", 1.0, dtype)
    for r in room:
        assert bool((r[n:] == 3.0).all())


def test_reproducible():
    for shape, gate_n in (((3, 20, 21, 22, 60), 3), ((2000, 1, 1, 2, 40), 2000), ((2, 30, 30, 30, 64), 1)):
        t, p = problem(shape, BF, gate_n=gate_n)
        g, q = {k: to_dev(v, BF) for k, v in t.items()}, dev(p)
        first = None
        for _ in range(3):
            got = cf.cf_resnorm_fwd(g["x"], g["f"], KIND["layer"], EPS, **q) + cf.cf_resnorm_bwd(
                g["f"], g["r"], g["dr"], g["dy"], KIND["layer"], EPS, **q)
            first = first or got
            assert all(torch.equal(a, b) for a, b in zip(got, first))


def test_gradient_against_differences():
    """The gradients as the derivative of the library's own forward, fp32,
    central differences along random directions of length 1, step h."""
    shape, h, alpha = (2, 2, 3, 2, 20), 2.0 ** -5, 0.8
    t, p = problem(shape, F32, gate_n=2)
    g, q = {k: to_dev(v, F32) for k, v in t.items()}, dev(p)
    names = list(q)

    def f(x, fb, *v):
        R, Y = cf.cf_resnorm_fwd(x, fb, KIND["layer"], EPS, alpha=alpha, **dict(zip(names, v)))
        return float((R.double() * g["dr"].double()).sum() + (Y.double() * g["dy"].double()).sum())

    args = [g["x"], g["f"]] + [q[n] for n in names]
    R, Y = cf.cf_resnorm_fwd(g["x"], g["f"], KIND["layer"], EPS, alpha=alpha, **q)
    got = dict(zip(("x", "f", "gpre", "bpre", "gpost", "bpost", "gate"),
                   cf.cf_resnorm_bwd(g["f"], R, g["dr"], g["dy"], KIND["layer"], EPS, alpha=alpha, **q)))
    size = float((R.double() * g["dr"].double()).abs().sum() + (Y.double() * g["dy"].double()).abs().sum())
    gen = torch.Generator(device="cuda").manual_seed(2)
    for k, (a, n) in enumerate(zip(args, ["x", "f"] + names)):
        e = torch.randn(a.shape, generator=gen, device="cuda")
        e = e / e.norm()
        at = lambda s: f(*[b + s * e if j == k else b for j, b in enumerate(args)])  # noqa: E731
        # truncation h^2 / 6 f''' (a direction of length 1 over rows of spread ~1: f''' below 100), rounding G size / h
        assert abs((at(h) - at(-h)) / (2 * h) - float((got[n].double() * e.double()).sum())) <= h * h / 6 * 100 + U * size / h


def test_past_2_31_elements():
    """64-bit offsets: rows behind 2^31 elements."""
    shape = (2, 129, 128, 129, 512)
    gen = torch.Generator(device="cuda").manual_seed(6)
    x, f = (torch.empty(shape, dtype=BF, device="cuda") for _ in range(2))
    for v in (x, f):
        for i in range(2):
            v[i] = torch.randn(shape[1:], generator=gen, device="cuda")
    ga, gate = torch.rand(512, generator=gen, device="cuda"), torch.rand(2, 512, generator=gen, device="cuda")
    R, Y = cf.cf_resnorm_fwd(x, f, KIND["rms"], EPS, gpre=ga, gpost=ga, gate=gate)
    dX, dF, *_ = cf.cf_resnorm_bwd(f, R, x, Y, KIND["rms"], EPS, gpre=ga, gpost=ga, gate=gate)
    at = slice(shape[1] - 1, shape[1])
    part = lambda v: v[1:, at].contiguous()  # noqa: E731
    R2, Y2 = cf.cf_resnorm_fwd(part(x), part(f), KIND["rms"], EPS, gpre=ga, gpost=ga, gate=gate[1])
    dX2, dF2, *_ = cf.cf_resnorm_bwd(part(f), part(R), part(x), part(Y), KIND["rms"], EPS, gpre=ga, gpost=ga, gate=gate[1])
    for whole, small in ((R, R2), (Y, Y2), (dX, dX2), (dF, dF2)):
        assert torch.equal(part(whole), small)
    t = {"x": host64(part(x)[:, :, :1, :4]), "f": host64(part(f)[:, :, :1, :4])}
    p = {"gpre": host64(ga), "gpost": host64(ga), "gate": host64(gate[1:])}
    check_fwd(part(R)[:, :, :1, :4], part(Y)[:, :, :1, :4], t, p, "rms", 1.0, BF)
