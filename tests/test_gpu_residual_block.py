"""A residual network over voxels as its user runs it: pointwise layers with the
activation and bias fused, the joins with their norms, the backward through all
of it, clipped gradients and Muon's update; on streams and in captured graphs."""
import numpy as np
import pytest
import torch

import oracle
import synthdata as sd
from cnn_cosmology_volumes_amd import cf
from gpu_util import host64, to_dev

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
EPS = 1e-5
LAYER, SILU = cf.CF_NORM_LAYER, cf.CF_ACT_SILU
BLOCKS, C, WIDE, SHAPE = 2, 24, 56, (3, 4, 3, 5)


def parameters(seed=0):
    rng = np.random.default_rng(seed)
    f = lambda *s: (rng.standard_normal(s)).astype(np.float32)  # noqa: E731
    v = lambda *s: rng.uniform(0.5, 1.5, s).astype(np.float32)  # noqa: E731
    return [{"w1": f(C, WIDE) / np.float32(np.sqrt(C)), "b1": 0.2 * f(WIDE), "w2": f(WIDE, C) / np.float32(np.sqrt(WIDE)),
             "b2": 0.2 * f(C), "gpre": v(C), "bpre": 0.2 * f(C), "gpost": v(C), "bpost": 0.2 * f(C),
             "gate": 0.5 * v(SHAPE[0], C)} for _ in range(BLOCKS)]


def step(p, x, y0, target, dtype):
    """x: the stream, y0: the first branch's input.  -> (loss gradient at the
    output, per-block gradients)."""
    kept, y = [], y0
    for q in p:
        w1, w2 = q["w1"].to(dtype), q["w2"].to(dtype)
        pre1, h = cf.cf_linear_fwd(y, w1, q["b1"], SILU)
        _, f = cf.cf_linear_fwd(h, w2, q["b2"], need_pre=False)
        r, y2 = cf.cf_resnorm_fwd(x, f, LAYER, EPS, q["gpre"], q["bpre"], q["gpost"], q["bpost"], q["gate"])
        kept.append((y, w1, w2, pre1, h, f, r))
        x, y = r, y2
    dy, dr = (y.float() - target).to(dtype), None
    grads = []
    for q, (yi, w1, w2, pre1, h, f, r) in zip(reversed(p), reversed(kept)):
        dx, df, *vec = cf.cf_resnorm_bwd(f, r, dr, dy, LAYER, EPS, q["gpre"], q["bpre"], q["gpost"], q["bpost"], q["gate"])
        dh, dw2, db2 = cf.cf_linear_bwd(h, w2, None, df)
        dy, dw1, db1 = cf.cf_linear_bwd(yi, w1, pre1, dh, SILU)
        dr = dx
        grads.insert(0, dict(zip(("w1", "b1", "w2", "b2", "gpre", "bpre", "gpost", "bpost", "gate"),
                                 [dw1, db1, dw2, db2, *vec])))
    return y, dr, dy, grads


def reference(p, x, y0, target):
    x, y = x.astype(np.float64), y0.astype(np.float64)
    kept = []
    for q in p:
        pre1, h = oracle.linear_fwd(y, q["w1"], q["b1"], "silu", 0.0)
        _, f = oracle.linear_fwd(h, q["w2"], q["b2"], "lrelu", 1.0)
        v = {k: q[k] for k in ("gpre", "bpre", "gpost", "bpost", "gate")}
        r, y2 = oracle.resnorm_fwd(x, f, "layer", EPS, **v)
        kept.append((y, pre1, h, f, r, v))
        x, y = r, y2
    dy, dr, grads = y - target, None, []
    for q, (yi, pre1, h, f, r, v) in zip(reversed(p), reversed(kept)):
        g = oracle.resnorm_bwd(f, r, dr, dy, "layer", EPS, **v)
        sh = yi.shape[:-1]
        dh, dw2, db2 = oracle.linear_bwd(h, q["w2"], np.zeros(sh + (C,)) + 1.0, g["df"], "lrelu", 1.0)
        dy, dw1, db1 = oracle.linear_bwd(yi, q["w1"], pre1, dh, "silu", 0.0)
        dr = g["dx"]
        grads.insert(0, {"w1": dw1, "b1": db1, "w2": dw2, "b2": db2, **{k: g["d" + k] for k in v}})
    return y, dr, dy, grads


def inputs(dtype, seed=1):
    rng = np.random.default_rng(seed)
    rnd = (lambda a: sd.bf16_round_f32(a.astype(np.float32))) if dtype == BF else (lambda a: a.astype(np.float32))
    return [rnd(rng.standard_normal(SHAPE + (C,))) for _ in range(2)] + [rng.standard_normal(SHAPE + (C,)).astype(np.float32)]


def rounded(p, dtype):
    if dtype != BF:
        return p
    return [{k: sd.bf16_round_f32(v) if k in ("w1", "w2") else v for k, v in q.items()} for q in p]


@pytest.mark.parametrize("dtype", [F32, BF], ids=["f32", "bf16"])
def test_network_of_two_blocks(dtype):
    p, (x, y0, target) = parameters(), inputs(dtype)
    y, dr, dy, grads = step([{k: to_dev(v, F32) for k, v in q.items()} for q in p], to_dev(x, dtype), to_dev(y0, dtype),
                            to_dev(target, F32), dtype)
    yo, dro, dyo, want = reference(rounded(p, dtype), x, y0, target)
    # Relative to each tensor's rms.  fp32: some 20 operations one after another, each off by at most some 32 u of
    # its terms, with gains below 10.  bf16: 12 tensors between them are rounded, 2^-8 each, and the norms' and
    # products' gains (weights of unit gain, gammas up to 1.5) multiply no more than 4 of them.
    tol = 1e-4 if dtype == F32 else 12 * 2.0 ** -8 * 4
    rel = lambda a, b: np.abs(host64(a) - b).max() / np.sqrt((b * b).mean())  # noqa: E731
    assert rel(y, yo) <= tol and rel(dr, dro) <= tol and rel(dy, dyo) <= tol
    for g, w in zip(grads, want):
        for k in w:
            assert rel(g[k], w[k]) <= tol, k


def train_step(p, mom, x, y0, target, dtype, max_norm):
    y, _, _, grads = step(p, x, y0, target, dtype)
    flat = [g[k] for g in grads for k in g]
    stats = cf.cf_grad_clip(flat, max_norm)
    cf.cf_muon(cf.muon_params(0.02), [q[k] for q in p for k in ("w1", "w2")], [g[k] for g in grads for k in ("w1", "w2")],
               mom)
    for q, g in zip(p, grads):
        for k in q:
            if k not in ("w1", "w2"):
                cf.cf_sgd(q[k], g[k], 0.01)
    return stats, flat


def test_clipped_step():
    """The clipped gradients of the whole network have the norm asked for, and the vectors move by them."""
    p, (x, y0, target) = parameters(), inputs(F32)
    d = [{k: to_dev(v, F32) for k, v in q.items()} for q in p]
    before = [{k: v.clone() for k, v in q.items()} for q in d]
    mom = [torch.zeros_like(q[k]) for q in d for k in ("w1", "w2")]
    stats, flat = train_step(d, mom, to_dev(x, F32), to_dev(y0, F32), to_dev(target, F32), F32, 0.5)
    want = reference(p, x, y0, target)[3]
    norm = np.sqrt(sum((g[k] ** 2).sum() for g in want for k in g))
    assert abs(stats[0].item() - norm) <= 1e-4 * norm and abs(stats[1].item() - 0.5 / norm) <= 1e-4 * 0.5 / norm
    assert abs(float(torch.cat([t.flatten() for t in flat]).double().norm()) - 0.5) <= 1e-6
    for q, b, g in zip(d, before, want):
        move = host64(b["gpre"]) - host64(q["gpre"])
        assert np.abs(move - 0.01 * 0.5 / norm * g["gpre"]).max() <= 1e-6


@pytest.mark.parametrize("dtype", [F32, BF], ids=["f32", "bf16"])
def test_captured_step(dtype):
    """The whole step in a graph, replayed between eager work: every replay gives
    the eager step's bits from the same state, with inputs that change."""
    p = parameters()
    make = lambda: [{k: to_dev(v, F32) for k, v in q.items()} for q in p]  # noqa: E731
    eager, graph = make(), make()
    momenta = lambda d: [torch.zeros_like(q[k]) for q in d for k in ("w1", "w2")]  # noqa: E731
    me, mg = momenta(eager), momenta(graph)
    buf = [to_dev(v, t) for v, t in zip(inputs(dtype), (dtype, dtype, F32))]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        warm = make()
        train_step(warm, momenta(warm), *buf, dtype, 0.5)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        stats, flat = train_step(graph, mg, *buf, dtype, 0.5)
    for i in range(4):
        for b, v, t in zip(buf, inputs(dtype, seed=10 + i), (dtype, dtype, F32)):
            b.copy_(to_dev(v, t))
        g.replay()
        s2, f2 = train_step(eager, me, *buf, dtype, 0.5)
        torch.cuda.synchronize()
        assert torch.equal(stats, s2) and all(torch.equal(a, b) for a, b in zip(flat, f2))
        assert all(torch.equal(a[k], b[k]) for a, b in zip(eager, graph) for k in a)


@pytest.mark.parametrize("dtype", [F32, BF], ids=["f32", "bf16"])
def test_two_streams_at_once(dtype):
    """Two steps on two streams, not ordered against each other, give what each gives alone."""
    p = parameters()
    make = lambda: [{k: to_dev(v, F32) for k, v in q.items()} for q in p]  # noqa: E731
    data = [[to_dev(v, t) for v, t in zip(inputs(dtype, s), (dtype, dtype, F32))] for s in (3, 4)]
    alone = []
    for d in data:
        q = make()
        alone.append(train_step(q, [torch.zeros_like(v[k]) for v in q for k in ("w1", "w2")], *d, dtype, 0.5))
    torch.cuda.synchronize()
    streams, got, nets = [torch.cuda.Stream(), torch.cuda.Stream()], [None, None], [make(), make()]
    moms = [[torch.zeros_like(v[k]) for v in q for k in ("w1", "w2")] for q in nets]
    torch.cuda.synchronize()
    for _ in range(3):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                q = [{k: v.clone() for k, v in b.items()} for b in nets[i]]
                got[i] = train_step(q, [m.clone() for m in moms[i]], *data[i], dtype, 0.5)
        torch.cuda.synchronize()
        for a, b in zip(got, alone):
            assert torch.equal(a[0], b[0]) and all(torch.equal(u, v) for u, v in zip(a[1], b[1]))


def test_stream_argument():
    """stream=: outputs in that stream's memory, whole once the streams are ordered."""
    x, y0, _ = (to_dev(v, BF) for v in inputs(BF))
    w = to_dev(parameters()[0]["w1"], BF)
    s = torch.cuda.Stream()
    want = cf.cf_linear_fwd(x, w, act=SILU)
    back = cf.cf_linear_bwd(x, w, want[0], want[1], SILU)
    join = cf.cf_resnorm_fwd(x, y0, LAYER, EPS)
    jback = cf.cf_resnorm_bwd(y0, join[0], x, y0, LAYER, EPS)
    g = [back[1].clone(), back[2].clone()]
    stats = cf.cf_grad_clip(g, 0.1)
    torch.cuda.synchronize()
    for _ in range(3):
        s.wait_stream(torch.cuda.current_stream())
        a = cf.cf_linear_fwd(x, w, act=SILU, stream=s)
        b = cf.cf_linear_bwd(x, w, a[0], a[1], SILU, stream=s)
        c = cf.cf_resnorm_fwd(x, y0, LAYER, EPS, stream=s)
        d = cf.cf_resnorm_bwd(y0, c[0], x, y0, LAYER, EPS, stream=s)
        st = cf.cf_grad_clip([b[1], b[2]], 0.1, stream=s)
        n = cf.cf_linear_fwd(x, w, act=SILU, need_pre=False, stream=s)
        torch.cuda.current_stream().wait_stream(s)
        assert n[0] is None and torch.equal(n[1], want[1])
        assert torch.equal(st, stats) and torch.equal(b[1], g[0]) and torch.equal(b[2], g[1])
        for u, v in zip(a + (b[0],) + c + d[:2], want + (back[0],) + join + jback[:2]):
            assert torch.equal(u, v)
