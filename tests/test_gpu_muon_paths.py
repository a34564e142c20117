"""Newton-Schulz and Muon at the sizes where the library changes its way of
computing: one block (shorter side up to 64, with or without the whole matrix
in LDS), fp64 rounds (tiles of 16, and of 32 from 449), split fp16 products
(from about 300 where the longer side is not much longer, with tiles of 64,
128 and 256 and reductions cut over blocks), and coefficients that the split
products do not take.

The reference is the definition in float64.  Tolerance as in
test_gpu_muon.py: |out - exact| <= 2^-22 K sum_k |a|^(steps - 1 - k) |X_k|,
K = |a| + 2 |b| + 4 |c| (Frobenius norms), and 2^-8 |out| for bf16."""
import pytest
import torch

from cnn_cosmology_volumes_amd import cf

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
NS = (5, 3.4445, -4.7750, 2.0315, 1e-7)


def reference(x, ns):
    """-> (result, tolerance) in float64."""
    steps, a, b, c, eps = ns
    t = x.double()
    if t.shape[0] > t.shape[1]:
        t = t.t()
    t = t.contiguous()
    t = t / (t.norm() + eps)
    k, tol = abs(a) + 2 * abs(b) + 4 * abs(c), 0.0
    for i in range(steps):
        tol += 2.0 ** -22 * k * abs(a) ** (steps - 1 - i) * t.norm().item()
        g = t @ t.t().contiguous()
        t = a * t + (b * g + c * (g @ g)) @ t
    return (t.t().contiguous() if x.shape[0] > x.shape[1] else t), tol


def gradient(seed, rows, cols, dtype=F32):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    r = min(4, rows, cols)
    u = torch.randn(rows, r, generator=gen, device="cuda") * 0.6 ** torch.arange(r, device="cuda")
    v = torch.randn(r, cols, generator=gen, device="cuda")
    return (1e-3 * (u @ v + torch.randn(rows, cols, generator=gen, device="cuda"))).to(dtype)


def check(got, x, ns=NS):
    want, tol = reference(x, ns)
    if x.dtype == BF:
        tol += 2.0 ** -8 * want.norm().item()
    err = (got.double() - want).norm().item()
    assert err <= tol, (tuple(x.shape), err, tol)


SHAPES = [(1, 1), (1, 640), (1, 641), (640, 16), (641, 16), (17, 208), (209, 17), (48, 208), (209, 48), (64, 64),
          (64, 128), (64, 129), (129, 64), (60, 3000), (5000, 33), (65, 65), (65, 4097), (128, 128), (2049, 192),
          (200, 319), (257, 255), (319, 319), (319, 640), (320, 320), (320, 9000), (7001, 333), (321, 352), (640, 511),
          (768, 2000), (448, 450), (449, 5001), (500, 4000), (7003, 600), (6000, 640), (1300, 1290), (2000, 1025), (2300, 2900), (4090, 4000)]


@pytest.mark.parametrize("dtype", [F32, BF], ids=["f32", "bf16"])
@pytest.mark.parametrize("shape", SHAPES, ids=["%dx%d" % s for s in SHAPES])
def test_newton_schulz(shape, dtype):
    x = gradient(sum(shape), *shape, dtype=dtype)
    check(cf.cf_newton_schulz(cf.newton_schulz_params(), [x])[0], x)


@pytest.mark.parametrize("ns", [(1,) + NS[1:], (2,) + NS[1:], (4,) + NS[1:], (7, 1.5, -0.5, 0.0, 1e-7),
                                (6, 2.0, -1.5, 0.5, 1e-7), (32, 1.875, -1.25, 0.375, 1e-7)])
@pytest.mark.parametrize("shape", [(20, 30), (64, 300), (300, 290), (400, 330), (1500, 2100)])
def test_steps_and_coefficients(shape, ns):
    x = gradient(9, *shape)
    check(cf.cf_newton_schulz(cf.newton_schulz_params(*ns), [x])[0], x, ns)


def test_coefficients_without_a_small_bound():
    """X grows past what the split fp16 products hold: the fp64 path computes
    Q in fp64, and s Q U with fp32 sums, each within 2^-21 of the terms'
    sizes, |Q|_F |s U|_F at most; the result is rounded once."""
    ns = (2, 20.0, -20.0, 1.0, 1e-7)
    x = gradient(3, 600, 530)
    out = cf.cf_newton_schulz(cf.newton_schulz_params(*ns), [x])[0]
    want, _ = reference(x, ns)
    t = x.double().t().contiguous()
    t = t / (t.norm() + ns[4])
    q = torch.eye(530, dtype=torch.float64, device="cuda")
    for _ in range(ns[0]):
        g = t @ t.t().contiguous()
        p = ns[1] * torch.eye(530, dtype=torch.float64, device="cuda") + ns[2] * g + ns[3] * (g @ g)
        q, t = p @ q, p @ t
    tol = 2.0 ** -21 * q.norm().item() + 2.0 ** -24 * want.norm().item()
    assert (out.double() - want).norm().item() <= tol


LISTS = [[(108, 32), (16, 16), (3, 200)], [(64, 300), (40, 50)], [(300, 64), (64, 3), (128, 1000)],
         [(2300, 2900), (108, 32), (64, 700), (300, 280), (500, 340)], [(330, 8000), (8000, 330)],
         [(400, 410), (440, 430)], [(400, 410), (32, 40), (700, 650)]]


@pytest.mark.parametrize("nesterov", [False, True])
@pytest.mark.parametrize("shapes", LISTS, ids=["-".join("%dx%d" % s for s in l) for l in LISTS])
def test_muon_of_lists(shapes, nesterov):
    """w (1 - lr wd) - lr f O(u): w's and the update's roundings, 2^-23 of
    their sizes, beside lr f times O's tolerance and what u's roundings, 2^-23
    |u|, become in O (as products' of relative error 2^-23 at the first step)."""
    lr, mu, wd = 0.0625, 0.875, 0.25      # exact in fp32
    hp = cf.muon_params(lr, momentum=mu, nesterov=nesterov, weight_decay=wd, scale=cf.CF_MUON_SCALE_RMS)
    gen = torch.Generator(device="cuda").manual_seed(4)
    w = [torch.randn(s, generator=gen, device="cuda") for s in shapes]
    g = [gradient(i, *s) for i, s in enumerate(shapes)]
    m = [4 * gradient(50 + i, *s) for i, s in enumerate(shapes)]
    w0, m0 = [t.double() for t in w], [t.double() for t in m]
    cf.cf_muon(hp, w, g, m)
    for i, s in enumerate(shapes):
        mo = mu * m0[i] + g[i].double()
        u = g[i].double() + mu * mo if nesterov else mo
        o, tol = reference(u, NS)
        f = 0.2 * max(s) ** 0.5
        wo = w0[i] * (1 - lr * wd) - lr * f * o
        assert torch.all((m[i].double() - mo).abs() <= 2.0 ** -23 * (mo.abs() + m0[i].abs()))
        tol = lr * f * (tol + 4 * 2.0 ** -23 * abs(NS[1]) ** 5) + 2.0 ** -22 * (w0[i].norm() + lr * f * o.norm()).item()
        assert (w[i].double() - wo).norm().item() <= tol, s


@pytest.mark.parametrize("shapes", [[(108, 32)], [(64, 300), (40, 50)], [(300, 64), (200, 280)], [(640, 511)], [(1500, 2100)],
                                    [(330, 8000)], [(2300, 2900)]], ids=str)
def test_nothing_is_read_from_the_workspace(shapes):
    """A workspace of NaNs, and one of other bytes, gives the same bits."""
    ns, x = cf.newton_schulz_params(), [gradient(i, *s) for i, s in enumerate(shapes)]
    size = cf.lib().cf_newton_schulz_workspace_size(cf.CF_F32, len(x), *cf._mat_sizes(x))
    got = []
    for fill in (0xFF, 0x7B, 0):
        ws = torch.full((size,), fill, dtype=torch.uint8, device="cuda")
        got.append(cf.cf_newton_schulz(ns, x, ws=ws))
    for other in got[1:]:
        for p, q in zip(got[0], other):
            assert torch.isfinite(p).all() and torch.equal(p, q)


@pytest.mark.parametrize("shape", [(20, 30), (64, 300), (300, 290), (400, 330), (1500, 2100)])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_a_bad_value_does_not_pass_unseen(shape, bad):
    x = gradient(2, *shape)
    x[3, 7] = bad
    out = cf.cf_newton_schulz(cf.newton_schulz_params(), [x])[0]
    assert torch.isnan(out[3, 7])


def test_own_stream_and_graph_of_large_matrices():
    ns, x = cf.newton_schulz_params(), [gradient(1, 1500, 2100), gradient(2, 400, 330)]
    a = cf.cf_newton_schulz(ns, x)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    b = cf.cf_newton_schulz(ns, x, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    for p, q in zip(a, b):
        assert torch.equal(p, q)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = cf.cf_newton_schulz(ns, x)
    for r in range(4):
        for t in x:
            t.copy_(t.flip(0).contiguous() * 0.5)
        graph.replay()
        eager = cf.cf_newton_schulz(ns, x)
        torch.cuda.synchronize()
        for p, q in zip(held, eager):
            assert torch.equal(p, q), r
