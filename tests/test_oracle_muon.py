"""The Newton-Schulz and Muon oracle against the singular value decomposition,
and the entry points' refusals (validation happens before any GPU work, so
these run without a GPU; pointers passed here are never dereferenced)."""
import ctypes

import numpy as np
import pytest
import torch

import oracle
from cnn_cosmology_volumes_amd import cf

NS = (5, 3.4445, -4.7750, 2.0315, 1e-7)
FAKE = 0x100000
MIS = 0x100008


@pytest.mark.parametrize("shape", [(1, 1), (5, 3), (3, 5), (8, 8), (40, 7)])
def test_each_singular_value_goes_through_the_polynomial(shape):
    x = np.random.default_rng(sum(shape)).standard_normal(shape)
    u, s, vt = np.linalg.svd(x, full_matrices=False)
    s = s / (np.sqrt(np.sum(s * s)) + NS[4])
    for _ in range(NS[0]):
        s = NS[1] * s + NS[2] * s ** 3 + NS[3] * s ** 5
    assert np.allclose(oracle.newton_schulz(x, *NS), (u * s) @ vt, rtol=0, atol=1e-10)


def test_cubic_iteration_converges_to_the_polar_factor():
    x = np.random.default_rng(1).standard_normal((6, 9)) + 2 * np.eye(6, 9)
    u, _, vt = np.linalg.svd(x, full_matrices=False)
    assert np.allclose(oracle.newton_schulz(x, 30, 1.5, -0.5, 0.0, 1e-12), u @ vt, atol=1e-8)


def test_muon_step_by_hand():
    w, g, m = np.array([[2.0, 0.0]]), np.array([[3.0, 4.0]]), np.array([[1.0, -1.0]])
    # one row: the factor is u / |u| times the polynomial's value at 1
    p = 1.0
    for _ in range(5):
        p = NS[1] * p + NS[2] * p ** 3 + NS[3] * p ** 5
    m1 = 0.5 * m + g
    u = g + 0.5 * m1
    want = w * (1 - 0.1 * 0.2) - 0.1 * np.sqrt(2.0) * p * u / np.sqrt(np.sum(u * u))
    got, mo = oracle.muon_step(w, g, m, 0.1, 0.5, True, 0.2, "aspect", NS)
    assert np.allclose(got, want, atol=1e-6) and np.array_equal(mo, m1)


def _arrays(shapes):
    k = len(shapes)
    return ((ctypes.c_int64 * k)(*[s[0] for s in shapes]), (ctypes.c_int64 * k)(*[s[1] for s in shapes]))


def _ptrs(k, v=FAKE):
    return (ctypes.c_void_p * k)(*[v] * k)


def _ns(shapes=((64, 32),), dt=cf.CF_F32, p=None, x=FAKE, out=FAKE, ws=ctypes.c_void_p(FAKE), wsb=1 << 40, k=None):
    rows, cols = _arrays(shapes)
    n = len(shapes) if k is None else k
    return cf.lib().cf_newton_schulz(ctypes.byref(p or cf.newton_schulz_params()), dt, n, rows, cols,
                                     _ptrs(len(shapes), x), _ptrs(len(shapes), out), ws, wsb, None)


def _muon(hp, shapes=((64, 32),), w=FAKE, g=FAKE, m=FAKE, wsb=1 << 40):
    rows, cols = _arrays(shapes)
    k = len(shapes)
    return cf.lib().cf_muon(ctypes.byref(hp), k, rows, cols, _ptrs(k, w), _ptrs(k, g), _ptrs(k, m),
                            ctypes.c_void_p(FAKE), wsb, None)


def test_refusals():
    inv, uns, wse = cf.CF_ERR_INVALID, cf.CF_ERR_UNSUPPORTED, cf.CF_ERR_WORKSPACE
    nan, inf = float("nan"), float("inf")
    assert _ns(dt=3) == inv
    assert _ns(shapes=((0, 4),)) == inv and _ns(shapes=((4, -1),)) == inv and _ns(shapes=((4, 4), (1 << 31, 1))) == inv
    assert _ns(shapes=((20000, 20000),)) == uns
    assert _ns(shapes=((4, 4),) * 33) == inv and _ns(k=0) == inv
    for p in (cf.newton_schulz_params(steps=0), cf.newton_schulz_params(steps=33), cf.newton_schulz_params(a=nan),
              cf.newton_schulz_params(c=inf), cf.newton_schulz_params(eps=0.0), cf.newton_schulz_params(eps=nan)):
        assert _ns(p=p) == inv
    assert _ns(x=0) == inv and _ns(x=MIS) == inv and _ns(out=0) == inv and _ns(out=MIS) == inv
    assert _ns(wsb=8) == wse and _ns(ws=None) == inv and _ns(ws=ctypes.c_void_p(MIS)) == inv
    assert b"workspace" in cf.lib().cf_last_error()
    for hp in (cf.muon_params(nan), cf.muon_params(0.1, momentum=1.0), cf.muon_params(0.1, momentum=-0.1),
               cf.muon_params(0.1, weight_decay=-1.0), cf.muon_params(0.1, weight_decay=inf),
               cf.muon_params(0.1, scale=2), cf.muon_params(0.1, ns=cf.newton_schulz_params(steps=0))):
        assert _muon(hp) == inv
    ok = cf.muon_params(0.1)
    assert _muon(ok, w=0) == inv and _muon(ok, g=MIS) == inv and _muon(ok, m=0) == inv and _muon(ok, wsb=8) == wse


def test_workspace_sizes():
    rows, cols = _arrays(((108, 32), (864, 64)))
    L = cf.lib()
    n = L.cf_newton_schulz_workspace_size(cf.CF_F32, 2, rows, cols)
    assert n > 0
    hp = cf.muon_params(0.1, nesterov=False)
    m0 = L.cf_muon_workspace_size(ctypes.byref(hp), 2, rows, cols)
    hp = cf.muon_params(0.1, nesterov=True)
    m1 = L.cf_muon_workspace_size(ctypes.byref(hp), 2, rows, cols)
    # Nesterov's direction is held in fp32 beside the momentum
    assert m0 == n and m1 >= n + 4 * (108 * 32 + 864 * 64)
    assert L.cf_newton_schulz_workspace_size(cf.CF_F32, 0, rows, cols) == 0
    assert L.cf_newton_schulz_workspace_size(9, 2, rows, cols) == 0


def test_binding_refuses_other_layouts():
    ns, hp = cf.newton_schulz_params(), cf.muon_params(0.1)
    x = torch.zeros(4, 6)
    with pytest.raises(ValueError):
        cf.cf_newton_schulz(ns, [])
    with pytest.raises(ValueError):
        cf.cf_newton_schulz(ns, [x.t()])
    with pytest.raises(ValueError):
        cf.cf_newton_schulz(ns, [x[0]])
    with pytest.raises(TypeError):
        cf.cf_newton_schulz(ns, [x, x.bfloat16()])
    with pytest.raises(TypeError):
        cf.cf_newton_schulz(ns, [x.double()])
    with pytest.raises(ValueError):
        cf.cf_newton_schulz(ns, [x], out=[torch.zeros(6, 4)])
    with pytest.raises(ValueError):
        cf.cf_muon(hp, [x], [x], [])
    with pytest.raises(ValueError):
        cf.cf_muon(hp, [x], [torch.zeros(6, 4)], [x])
    with pytest.raises(TypeError):
        cf.cf_muon(hp, [x.bfloat16()], [x], [x])
