"""The oracle of linear layers, residual joins and gradient clipping against
central differences of its own forwards, and the entry points' refusals
(validation happens before any GPU work, so these run without a GPU; pointers
passed here are never dereferenced: every call fails)."""
import ctypes

import numpy as np
import pytest
import torch

import oracle
from cnn_cosmology_volumes_amd import cf

FAKE = ctypes.c_void_p(0x100000)
MIS = ctypes.c_void_p(0x100008)
INF, NAN = float("inf"), float("nan")
BF = torch.bfloat16


def differences(f, arrays, grads, rng, h=1e-5, tol=1e-6):
    """Central differences of the scalar f(*arrays) at a few places of each:
    truncation h^2 f'''/6 and cancellation 2^-52 |f| / h are both below 1e-8 here."""
    for k, (a, g) in enumerate(zip(arrays, grads)):
        for i in rng.choice(a.size, min(8, a.size), replace=False):
            e = np.zeros(a.size)
            e[i] = h
            e = e.reshape(a.shape)
            at = lambda s: f(*[b + s * e if j == k else b for j, b in enumerate(arrays)])  # noqa: E731
            assert abs((at(1) - at(-1)) / (2 * h) - np.asarray(g).flat[i]) < tol


@pytest.mark.parametrize("act", ["lrelu", "silu"])
def test_linear_backward_is_the_forwards_derivative(act):
    rng = np.random.default_rng(1)
    x, w, b = rng.standard_normal((7, 5)), rng.standard_normal((5, 3)), rng.standard_normal(3)
    dy, r = rng.standard_normal((7, 3)), rng.standard_normal((7, 3))
    f = lambda x, w, b: float((oracle.linear_fwd(x, w, b, act, 0.3, r)[1] * dy).sum())  # noqa: E731
    pre, _ = oracle.linear_fwd(x, w, b, act, 0.3, r)
    assert np.abs(pre).min() > 1e-3                  # no point near the leaky ReLU's kink
    differences(f, [x, w, b], oracle.linear_bwd(x, w, pre, dy, act, 0.3), rng)


@pytest.mark.parametrize("post", [False, True])
@pytest.mark.parametrize("gate_n", [0, 1, 2])
@pytest.mark.parametrize("kind", ["rms", "layer"])
def test_resnorm_backward_is_the_forwards_derivative(kind, gate_n, post):
    rng = np.random.default_rng(2)
    shape, eps, alpha = (2, 1, 3, 2, 6), 1e-3, 0.8
    x, f, wr, wy = (rng.standard_normal(shape) + 0.3 for _ in range(4))
    names = ["gpre", "bpre"] + (["gpost", "bpost"] if post else []) + (["gate"] if gate_n else [])
    vecs = {n: rng.uniform(0.5, 1.5, (gate_n, 6) if n == "gate" else 6) for n in names}

    def total(x, f, *v):
        r, y = oracle.resnorm_fwd(x, f, kind, eps, alpha=alpha, **dict(zip(names, v)))
        return float((r * wr).sum() + (y * wy).sum())

    r, _ = oracle.resnorm_fwd(x, f, kind, eps, alpha=alpha, **vecs)
    g = oracle.resnorm_bwd(f, r, wr, wy, kind, eps, alpha=alpha, **vecs)
    differences(total, [x, f] + [vecs[n] for n in names], [g["dx"], g["df"]] + [g["d" + n] for n in names], rng)


def test_clipped_gradients_have_the_norm():
    rng = np.random.default_rng(3)
    g = [rng.standard_normal(n) for n in (1, 17, 300)]
    out, norm, factor = oracle.grad_clip(g, 2.5)
    assert abs(np.linalg.norm(np.concatenate(out)) - 2.5) < 1e-12 and factor < 1
    assert oracle.grad_clip(g, norm * 1.01)[2] == 1.0


# ----------------------------------------------------------------- refusals
def lin_fwd(dt=cf.CF_BF16, rows=100, fin=64, fout=32, X=0x1000000, W=0x2000000, bias=0x3000000, act=cf.CF_ACT_SILU,
            slope=0.0, R=0x4000000, pre=0x5000000, Y=0x6000000, ws=0x7000000, wsb=1 << 20):
    return cf.lib().cf_linear_fwd(dt, rows, fin, fout, X, W, bias, act, slope, R, pre, Y, ws, wsb, None)


def lin_bwd(dt=cf.CF_BF16, rows=100, fin=64, fout=32, X=0x1000000, W=0x2000000, pre=0x3000000, dY=0x4000000,
            act=cf.CF_ACT_SILU, slope=0.0, dX=0x5000000, dW=0x6000000, db=0x7000000, ws=0x8000000, wsb=1 << 24):
    return cf.lib().cf_linear_bwd(dt, rows, fin, fout, X, W, pre, dY, act, slope, dX, dW, db, ws, wsb, None)


LINEAR_BAD = [dict(dt=7), dict(rows=0), dict(rows=-1), dict(fin=0), dict(fout=0), dict(fin=65537), dict(fout=1 << 20),
              dict(rows=(1 << 30) + 1), dict(rows=1 << 30, fin=4096), dict(X=None), dict(W=None), dict(X=0x1000008),
              dict(W=0x2000002), dict(act=2), dict(act=-1), dict(act=cf.CF_ACT_LRELU, slope=-0.1),
              dict(act=cf.CF_ACT_LRELU, slope=NAN), dict(act=cf.CF_ACT_LRELU, slope=INF)]


@pytest.mark.parametrize("kw", LINEAR_BAD + [dict(Y=None), dict(Y=0x6000008), dict(pre=0x5000004), dict(R=0x4000001),
                                             dict(bias=0x3000004)], ids=str)
def test_linear_fwd_refuses(kw):
    assert lin_fwd(**kw) == cf.CF_ERR_INVALID


@pytest.mark.parametrize("kw", LINEAR_BAD + [dict(dY=None), dict(dW=None), dict(pre=None), dict(db=0x7000004),
                                             dict(dX=0x5000008),
                                             dict(pre=None, act=cf.CF_ACT_LRELU, slope=0.5)], ids=str)
def test_linear_bwd_refuses(kw):
    assert lin_bwd(**kw) == cf.CF_ERR_INVALID


def test_linear_workspaces():
    size = lambda *a: int(cf.lib().cf_linear_workspace_size(*a))  # noqa: E731
    assert size(cf.CF_F32, 0, 4, 4, 0) == 0 and size(5, 4, 4, 4, 0) == 0 and size(cf.CF_F32, 4, 4, 70000, 1) == 0
    need = size(cf.CF_BF16, 24, 16384, 128, 0)         # a long reduction: split
    assert need > 0
    assert lin_fwd(rows=24, fin=16384, fout=128, wsb=need - 1) == cf.CF_ERR_WORKSPACE
    assert lin_fwd(rows=24, fin=16384, fout=128, wsb=need, ws=None) == cf.CF_ERR_INVALID
    assert lin_fwd(rows=24, fin=16384, fout=128, wsb=need, ws=0x7000008) == cf.CF_ERR_INVALID
    need = size(cf.CF_BF16, 100, 64, 32, 1)
    assert need >= 2 * 2 * 100 * 32                    # the gated gradient in two parts
    assert lin_bwd(wsb=need - 1) == cf.CF_ERR_WORKSPACE
    assert lin_bwd(wsb=need, ws=None) == cf.CF_ERR_INVALID


def refused(status):
    assert status == cf.CF_ERR_INVALID
    assert b"overlap" in cf.lib().cf_last_error()


def test_linear_overlaps():
    xb, wb, yb = 100 * 64 * 2, 64 * 32 * 2, 100 * 32 * 2
    for other in (0x1000000, 0x1000000 + xb - 16, 0x2000000 + wb - 16, 0x3000000, 0x4000000, 0x4000000 + yb - 16):
        refused(lin_fwd(Y=other))
        refused(lin_fwd(pre=other))
    refused(lin_fwd(pre=0x6000000))
    # a reduction that is split: its workspace counts
    refused(lin_fwd(rows=24, fin=16384, fout=128, R=None, ws=0x2000000 + (4 << 20) - 16, Y=0x9000000, wsb=1 << 30))
    for other in (0x1000000, 0x2000000 + wb - 16, 0x3000000, 0x4000000 + yb - 16):
        for name in ("dX", "dW", "db", "ws"):
            refused(lin_bwd(**{name: other}))
    refused(lin_bwd(dX=0x6000000))
    refused(lin_bwd(db=0x6000000 + 64 * 32 * 4 - 16))
    refused(lin_bwd(ws=0x6000000))


SHAPE = (2, 4, 4, 4, 32)


def params(kind=cf.CF_NORM_RMS, eps=1e-5, alpha=1.0, gpre=0x10000, bpre=0x11000, gpost=0x12000, bpost=0x13000,
           gate=0x14000, gate_n=2):
    return cf.cf_resnorm_params(kind, eps, alpha, gpre, bpre, gpost, bpost, gate, gate_n)


def res_fwd(dt=cf.CF_F32, shape=SHAPE, p=None, X=0x1000000, F=0x2000000, R=0x3000000, Y=0x4000000, **kw):
    p = ctypes.byref(params(**kw)) if p is None else p
    return cf.lib().cf_resnorm_fwd(dt, cf.dims(shape), p, X, F, R, Y, None)


def res_bwd(dt=cf.CF_F32, shape=SHAPE, F=0x1000000, R=0x2000000, dR=0x3000000, dY=0x4000000, dX=0x5000000,
            dF=0x6000000, grads=(0x7000000, 0x7001000, 0x7002000, 0x7003000, 0x7004000), ws=0x8000000, wsb=1 << 24, **kw):
    return cf.lib().cf_resnorm_bwd(dt, cf.dims(shape), ctypes.byref(params(**kw)), F, R, dR, dY, dX, dF, *grads, ws, wsb,
                                   None)


RES_BAD = [dict(dt=3), dict(shape=(0, 4, 4, 4, 32)), dict(shape=(2, 4, 4, -4, 32)), dict(kind=2), dict(eps=0.0),
           dict(eps=-1.0), dict(eps=NAN), dict(eps=INF), dict(alpha=NAN), dict(alpha=INF), dict(gate=None),
           dict(gate_n=0), dict(gate_n=3), dict(gate_n=-1), dict(gpost=None), dict(gpre=0x10008), dict(bpost=0x13004),
           dict(gate=0x14008), dict(F=None)]


@pytest.mark.parametrize("kw", RES_BAD + [dict(X=None), dict(R=None), dict(R=0x3000008), dict(Y=0x4000004),
                                          dict(p=ctypes.POINTER(cf.cf_resnorm_params)())], ids=str)
def test_resnorm_fwd_refuses(kw):
    assert res_fwd(**kw) == cf.CF_ERR_INVALID


@pytest.mark.parametrize("kw", RES_BAD + [dict(R=None), dict(dX=None), dict(dF=None), dict(dR=None, dY=None),
                                          dict(grads=(0x7000000, 0, 0, 0, None)), dict(grads=(0x7000004, 0, 0, 0, 0x7004000)),
                                          dict(ws=None), dict(ws=0x8000008)], ids=str)
def test_resnorm_bwd_refuses(kw):
    assert res_bwd(**kw) == cf.CF_ERR_INVALID


def test_resnorm_limits():
    assert res_fwd(shape=(1, 1, 1, 1, 4097), gate=None, gate_n=0) == cf.CF_ERR_UNSUPPORTED
    need = cf.cf_resnorm_workspace_size(cf.CF_F32, SHAPE, 2)
    assert need > 0 and res_bwd(wsb=need - 1) == cf.CF_ERR_WORKSPACE
    assert cf.cf_resnorm_workspace_size(cf.CF_F32, SHAPE, 3) == 0
    assert cf.cf_resnorm_workspace_size(cf.CF_F32, (1, 1, 1, 1, 4097), 0) == 0


def test_resnorm_overlaps():
    b = 2 * 64 * 32 * 4
    for other in (0x1000000, 0x1000000 + b - 16, 0x2000000 + b - 16, 0x10000, 0x14000 + 128):
        refused(res_fwd(R=other))
        refused(res_fwd(Y=other))
    refused(res_fwd(Y=0x3000000))
    for other in (0x1000000, 0x2000000 + b - 16, 0x3000000, 0x4000000, 0x12000):
        refused(res_bwd(dX=other))
        refused(res_bwd(dF=other))
        refused(res_bwd(ws=other))
        refused(res_bwd(grads=(other, 0, 0, 0, 0x7004000)))
    refused(res_bwd(dX=0x6000000))
    refused(res_bwd(grads=(0x7000000, 0x7000000 + 112, 0, 0, 0x7004000)))
    refused(res_bwd(grads=(0, 0, 0, 0x7004000 + 128, 0x7004000)))


def clip(sizes=(1000, 17, 4), dt=cf.CF_F32, g=(0x1000000, 0x2000000, 0x3000000), out=(0x4000000, 0x5000000, 0x6000000),
         max_norm=1.0, stats=0x7000000, ws=0x8000000, wsb=1 << 20, count=None):
    n = (ctypes.c_int64 * len(sizes))(*sizes)
    arr = lambda v: None if v is None else (ctypes.c_void_p * len(v))(*v)  # noqa: E731
    return cf.lib().cf_grad_clip(dt, len(sizes) if count is None else count, n, arr(g), arr(out), max_norm, stats, ws, wsb,
                                 None)


@pytest.mark.parametrize("kw", [dict(dt=2), dict(sizes=(1000, 0, 4)), dict(sizes=(1000, -1, 4)), dict(count=0),
                                dict(count=1025), dict(g=None), dict(g=(0x1000000, 0, 0x3000000)),
                                dict(g=(0x1000000, 0x2000008, 0x3000000)), dict(out=(0x4000000, 0, 0x6000000)),
                                dict(max_norm=-1.0), dict(max_norm=NAN), dict(stats=0x7000004), dict(ws=None),
                                dict(ws=0x8000008), dict(sizes=(1 << 37, 17, 4))], ids=str)
def test_clip_refuses(kw):
    assert clip(**kw) == cf.CF_ERR_INVALID


def test_clip_workspace():
    n = (ctypes.c_int64 * 1)(1000)
    need = int(cf.lib().cf_grad_clip_workspace_size(cf.CF_F32, 1, n))
    assert need > 0
    assert clip(sizes=(1000,), g=(0x1000000,), out=None, wsb=need - 1) == cf.CF_ERR_WORKSPACE
    assert int(cf.lib().cf_grad_clip_workspace_size(cf.CF_F32, 0, n)) == 0


def test_clip_overlaps():
    g = (0x1000000, 0x2000000, 0x3000000)
    refused(clip(out=(g[1], 0x5000000, 0x6000000)))                         # another's input
    refused(clip(out=(0x4000000, 0x5000000, g[0] + 3984)))                  # the last 16 bytes
    refused(clip(out=(g[0] + 16, 0x5000000, 0x6000000)))                    # its own, shifted
    refused(clip(out=(0x4000000, 0x4000000, 0x6000000)))                    # one output twice
    refused(clip(out=None, g=(g[0], g[0], g[2])))                           # one gradient twice, in place
    refused(clip(stats=g[0]))
    refused(clip(stats=0x4000000 + 16))
    refused(clip(ws=g[1]))
    refused(clip(ws=0x7000000))


# ----------------------------------------------------------------- bindings
def test_bindings_refuse_types_shapes_and_strides():
    x, w = torch.zeros(6, 8), torch.zeros(8, 4)
    y = torch.zeros(6, 4)
    for bad, error, match in [(dict(bias=torch.zeros(4, dtype=BF)), TypeError, "bias"),
                              (dict(bias=torch.zeros(8)), ValueError, "bias"), (dict(R=torch.zeros(6, 8)), ValueError, "R"),
                              (dict(Y=torch.zeros(6, 4, dtype=BF)), TypeError, "Y"),
                              (dict(pre=torch.zeros(4, 6).t()), ValueError, "pre"),
                              (dict(ws=torch.zeros(64, dtype=torch.uint8)[::2]), ValueError, "ws")]:
        with pytest.raises(error, match=match):
            cf.cf_linear_fwd(x, w, **bad)
    with pytest.raises(ValueError, match="W"):
        cf.cf_linear_fwd(x, torch.zeros(7, 4))
    with pytest.raises(ValueError, match="W"):
        cf.cf_linear_fwd(x, torch.zeros(4, 8).t())
    with pytest.raises(TypeError, match="W"):
        cf.cf_linear_fwd(x, w.to(BF))
    with pytest.raises(ValueError, match="X"):
        cf.cf_linear_fwd(torch.zeros(8, 6).t(), w)
    with pytest.raises(ValueError, match="dY"):
        cf.cf_linear_bwd(x, w, y, torch.zeros(6, 5))
    with pytest.raises(TypeError, match="dW"):
        cf.cf_linear_bwd(x, w, y, y, dW=torch.zeros(8, 4, dtype=BF))
    with pytest.raises(ValueError, match="db"):
        cf.cf_linear_bwd(x, w, y, y, db=torch.zeros(5))
    v, p = torch.zeros(2, 2, 2, 2, 8), torch.zeros(8)
    for bad, error, match in [(dict(gpre=torch.zeros(7)), ValueError, "gpre"), (dict(gate=torch.zeros(2, 7)), ValueError, "gate"),
                              (dict(gpost=p.to(BF)), TypeError, "gpost"), (dict(R=torch.zeros(2, 2, 2, 2, 4)), ValueError, "R"),
                              (dict(Y=v.transpose(1, 2)[:, :, :, :, ::1].transpose(0, 4)), ValueError, "Y")]:
        with pytest.raises(error, match=match):
            cf.cf_resnorm_fwd(v, v, cf.CF_NORM_RMS, 1e-5, **bad)
    with pytest.raises(ValueError, match="F"):
        cf.cf_resnorm_fwd(v, v[:1], cf.CF_NORM_RMS, 1e-5)
    with pytest.raises(TypeError, match="dY"):
        cf.cf_resnorm_bwd(v, v, v, v.to(BF), cf.CF_NORM_RMS, 1e-5)
    with pytest.raises(ValueError, match="empty"):
        cf.cf_grad_clip([], 1.0)
    with pytest.raises(TypeError, match="gradient 1"):
        cf.cf_grad_clip([p, p.to(BF)], 1.0)
    with pytest.raises(ValueError, match="output 0"):
        cf.cf_grad_clip([p], 1.0, out=[torch.zeros(7)])
    with pytest.raises(ValueError, match="stats"):
        cf.cf_grad_clip([p], 1.0, stats=torch.zeros(3))
    with pytest.raises(TypeError):
        cf.cf_grad_clip([p.double()], 1.0)


def _host_calls():
    x, w, v, p = torch.zeros(6, 8), torch.zeros(8, 4), torch.zeros(2, 2, 2, 2, 8), torch.zeros(8)
    y = torch.zeros(6, 4)
    return {"linear_fwd": lambda: cf.cf_linear_fwd(x, w), "linear_bwd": lambda: cf.cf_linear_bwd(x, w, y, y),
            "resnorm_fwd": lambda: cf.cf_resnorm_fwd(v, v, 0, 1e-5, p),
            "resnorm_bwd": lambda: cf.cf_resnorm_bwd(v, v, v, v, 0, 1e-5, p), "clip": lambda: cf.cf_grad_clip([x, w], 1.0)}


@pytest.mark.parametrize("name", sorted(_host_calls()))
def test_host_tensors(name):
    """A host address must not reach a kernel."""
    with pytest.raises(ValueError, match="GPU"):
        _host_calls()[name]()


ARGS = ["x", "w", "bias", "r", "pre", "y", "dx", "dw", "db", "f", "gpre", "bpost", "gate", "g1", "o1", "stats", "ws"]


@pytest.mark.parametrize("where", ARGS)
def test_one_tensor_elsewhere(where):
    """Each argument is looked at, not the first one alone.  (A stand-in for
    the GPU's index lets the checks run on any machine.)"""
    class Here(torch.Tensor):
        def get_device(self):
            return 0

    def t(name, *shape, dtype=torch.float32):
        a = torch.zeros(*shape, dtype=dtype)
        return a if name == where else a.as_subclass(Here)

    x, w, ws = t("x", 6, 8), t("w", 8, 4), t("ws", 1 << 16, dtype=torch.uint8)
    if where in ("x", "w", "bias", "r", "pre", "y", "ws"):
        with pytest.raises(ValueError, match="GPU"):
            cf.cf_linear_fwd(x, w, t("bias", 4), R=t("r", 6, 4), pre=t("pre", 6, 4), Y=t("y", 6, 4), ws=ws)
    if where in ("x", "w", "pre", "y", "dx", "dw", "db", "ws"):
        with pytest.raises(ValueError, match="GPU"):
            cf.cf_linear_bwd(x, w, t("pre", 6, 4), t("y", 6, 4), dX=t("dx", 6, 8), dW=t("dw", 8, 4), db=t("db", 4), ws=ws)
    shape = (2, 2, 2, 2, 8)
    vec = dict(gpre=t("gpre", 8), gpost=t("", 8), bpost=t("bpost", 8), gate=t("gate", 2, 8))
    if where in ("x", "f", "r", "y", "gpre", "bpost", "gate"):
        with pytest.raises(ValueError, match="GPU"):
            cf.cf_resnorm_fwd(t("x", *shape), t("f", *shape), 0, 1e-5, R=t("r", *shape), Y=t("y", *shape), **vec)
    if where in ("f", "r", "y", "dx", "gpre", "bpost", "gate", "ws"):
        with pytest.raises(ValueError, match="GPU"):
            cf.cf_resnorm_bwd(t("f", *shape), t("r", *shape), None, t("y", *shape), 0, 1e-5, dX=t("dx", *shape), ws=ws,
                              **vec)
    if where in ("g1", "o1", "stats", "ws"):
        with pytest.raises(ValueError, match="GPU"):
            cf.cf_grad_clip([t("", 4), t("g1", 5)], 1.0, out=[t("", 4), t("o1", 5)], stats=t("stats", 2), ws=ws)


def test_bindings_refuse_sizes_past_32_bits():
    """2^32 + 8 would be 8 to the library."""
    big, bf = (1 << 32) + 8, torch.bfloat16
    new = lambda *shape: torch.empty(shape, dtype=bf, device="meta")
    with pytest.raises(ValueError, match="too large"):
        cf.cf_linear_fwd(new(1, big), new(big, 8))
    with pytest.raises(ValueError, match="too large"):
        cf.cf_linear_bwd(new(1, 8), new(8, big), None, new(1, big))
    x = new(1, 1, 1, big, 1)
    with pytest.raises(ValueError, match="NDHWC"):
        cf.cf_resnorm_fwd(x, x, cf.CF_NORM_RMS, 1e-6)
    with pytest.raises(ValueError, match="NDHWC"):
        cf.cf_resnorm_bwd(x, x, x, x, cf.CF_NORM_RMS, 1e-6)
    flat = new(4, 8)
    with pytest.raises(ValueError, match="NDHWC"):
        cf.cf_resnorm_fwd(flat, flat, cf.CF_NORM_RMS, 1e-6)
