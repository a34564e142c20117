"""Group norm, Newton-Schulz and Muon refuse arguments that overlap what they
write (validation happens before any GPU work, so these run without a GPU;
addresses passed here are never dereferenced: every call fails)."""
import ctypes

import pytest

from cnn_cosmology_volumes_amd import cf

WS = 1 << 44                       # far from everything else
WSB = 1 << 34


def at(k):
    """Addresses 1 MiB apart; the matrices and tensors below are smaller."""
    return (k + 1) << 20


def arrays(shapes):
    k = len(shapes)
    return ((ctypes.c_int64 * k)(*[s[0] for s in shapes]), (ctypes.c_int64 * k)(*[s[1] for s in shapes]))


def ptrs(v):
    return (ctypes.c_void_p * len(v))(*v)


SHAPES = [(64, 32), (30, 50), (128, 8)]
BYTES = [4 * r * c for r, c in SHAPES]


def ns(x, out, ws=WS, dt=cf.CF_F32):
    rows, cols = arrays(SHAPES)
    p = cf.newton_schulz_params()
    return cf.lib().cf_newton_schulz(ctypes.byref(p), dt, len(SHAPES), rows, cols, ptrs(x), ptrs(out), ws, WSB, None)


def muon(w, g, m, ws=WS):
    rows, cols = arrays(SHAPES)
    hp = cf.muon_params(0.1)
    return cf.lib().cf_muon(ctypes.byref(hp), len(SHAPES), rows, cols, ptrs(w), ptrs(g), ptrs(m), ws, WSB, None)


A, B, C = [at(0), at(1), at(2)], [at(3), at(4), at(5)], [at(6), at(7), at(8)]


def swap(v, i, p):
    return v[:i] + [p] + v[i + 1:]


def refused(status):
    assert status == cf.CF_ERR_INVALID
    assert b"overlap" in cf.lib().cf_last_error()


def test_newton_schulz_in_place():
    refused(ns(A, A))


@pytest.mark.parametrize("i", range(3))
def test_newton_schulz(i):
    refused(ns(A, swap(B, i, A[(i + 1) % 3])))                                       # another matrix's input
    refused(ns(A, swap(B, i, A[i] + BYTES[i] - 16)))                                 # the last 16 bytes
    refused(ns(A, swap(B, i, B[(i + 1) % 3])))                                       # another matrix's output
    refused(ns(A, B, ws=A[i]))
    refused(ns(A, B, ws=B[i] + BYTES[i] - 16))


@pytest.mark.parametrize("i", range(3))
def test_muon(i):
    j = (i + 1) % 3
    refused(muon(A, swap(B, i, A[i]), C))
    refused(muon(A, B, swap(C, i, A[i])))
    refused(muon(A, B, swap(C, i, B[j])))
    refused(muon(swap(A, i, A[j]), B, C))                                            # a weight twice
    refused(muon(A, B, swap(C, i, C[j] + BYTES[j] - 16)))
    refused(muon(A, B, C, ws=B[i]))


SHAPE, GROUPS = (2, 4, 4, 4, 32), 4              # 16 KiB
P = {n: at(i) for i, n in enumerate(("X", "dY", "gamma", "beta", "mean", "rstd", "Y", "dX", "dgamma", "dbeta"))}
BIG = (1, 64, 64, 64, 32)                        # takes a workspace


def fwd(shape=SHAPE, ws=WS, **kw):
    p = dict(P, **kw)
    return cf.lib().cf_groupnorm_fwd(cf.CF_F32, cf.dims(shape), p["X"], GROUPS, p["gamma"], p["beta"], 1e-5,
                                     cf.CF_ACT_SILU, 0.0, p["Y"], p["mean"], p["rstd"], ws, WSB, None)


def bwd(shape=SHAPE, ws=WS, **kw):
    p = dict(P, **kw)
    return cf.lib().cf_groupnorm_bwd(cf.CF_F32, cf.dims(shape), p["X"], p["dY"], GROUPS, p["gamma"], p["beta"], p["mean"],
                                     p["rstd"], cf.CF_ACT_SILU, 0.0, p["dX"], p["dgamma"], p["dbeta"], ws, WSB, None)


def test_groupnorm():
    refused(fwd(Y=P["X"]))
    refused(fwd(Y=P["X"] + 4 * 2 * 64 * 32 - 16))
    refused(fwd(mean=P["gamma"]))
    refused(fwd(rstd=P["mean"]))
    refused(fwd(mean=P["Y"] + 64))
    refused(bwd(dX=P["X"]))
    refused(bwd(dX=P["dY"]))
    refused(bwd(dX=P["dY"] - 4 * 2 * 64 * 32 + 16))
    refused(bwd(dgamma=P["gamma"]))
    refused(bwd(dbeta=P["dgamma"] + 112))
    refused(bwd(dbeta=P["mean"]))
    # 32 MiB tensors, further apart
    far = {n: i << 32 for i, n in enumerate(("X", "dY", "gamma", "beta", "mean", "rstd", "Y", "dX", "dgamma", "dbeta"), 1)}
    refused(fwd(shape=BIG, ws=far["X"] + (1 << 20), **far))
    refused(bwd(shape=BIG, ws=far["dX"] + (1 << 20), **far))
