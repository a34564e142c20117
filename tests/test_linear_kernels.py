"""Every kernel of the linear layers' products: each type, product, tile, with the
reduction whole and split, at sizes with tiles inside the result and tiles that its
edges cut.  That the sizes reach the kernels is looked at without a GPU, so that
another estimate of tiles cannot leave one untested.

The oracle is elementary torch in 64 bits on the GPU.  Tolerances are those of
test_gpu_linear.py, and for dX of test_gpu_linear_digits.py (u = 2^-24): (K + 2) u of the sum
of a product's magnitudes and the terms' own errors; bf16 outputs add 2^-8 of the value."""
import pytest
import torch

from cnn_cosmology_volumes_amd import cf
from test_linear_tiles import DW, DW_ONE, DW_TWO, DX, FWD, FWD_RES, tiles

BF, F32 = torch.bfloat16, torch.float32
U, TINY = 2.0 ** -24, 1e-37
T64, T128, T256X128, T256 = (64, 64), (128, 128), (256, 128), (256, 256)
NAMES = ["fwd", "dX", "dW", "dW_one", "dW_two", "fwd_res"]

# type, product, tile, whether the reduction is split: rows, in, out
CASES = {
    (F32, FWD, T64, False): (107, 204, 104), (F32, FWD, T64, True): (101, 248, 106),
    (F32, FWD, T128, False): (12307, 241, 196), (F32, FWD, T128, True): (3745, 4981, 205),
    (F32, FWD, T256X128, False): (54546, 100, 197), (F32, FWD, T256X128, True): (15315, 6949, 193),
    (F32, FWD_RES, T64, False): (103, 101, 77), (F32, FWD_RES, T64, True): (100, 242, 78),
    (F32, FWD_RES, T128, False): (32602, 101, 202), (F32, FWD_RES, T128, True): (3916, 7281, 197),
    (F32, FWD_RES, T256X128, False): (41954, 580, 323), (F32, FWD_RES, T256X128, True): (30977, 7629, 194),
    (F32, DX, T64, False): (101, 104, 231), (F32, DX, T64, True): (106, 103, 247),
    (F32, DX, T128, False): (9804, 257, 242), (F32, DX, T128, True): (3723, 194, 4846),
    (F32, DX, T256X128, False): (54205, 204, 100), (F32, DX, T256X128, True): (15420, 198, 6133),
    (F32, DW, T64, False): (205, 106, 101), (F32, DW, T64, True): (243, 104, 105),
    (F32, DW, T128, False): (113, 8361, 324), (F32, DW, T128, True): (5517, 258, 582),
    (F32, DW_ONE, T64, False): (205, 106, 101), (F32, DW_ONE, T64, True): (243, 104, 105),
    (F32, DW_ONE, T128, False): (251, 8200, 329), (F32, DW_ONE, T128, True): (76306, 196, 196),
    (F32, DW_ONE, T256X128, False): (100, 2051, 6575), (F32, DW_ONE, T256X128, True): (48933, 1921, 193),
    (BF, FWD, T64, False): (107, 204, 104), (BF, FWD, T64, True): (102, 742, 106),
    (BF, FWD, T128, False): (16325, 168, 193), (BF, FWD, T128, True): (1564, 4849, 195),
    (BF, FWD, T256X128, False): (33171, 132, 154), (BF, FWD, T256X128, True): (25082, 8746, 129),
    (BF, FWD, T256, False): (29378, 131, 389), (BF, FWD, T256, True): (6699, 8574, 393),
    (BF, DX, T64, False): (101, 104, 231), (BF, DX, T64, True): (102, 108, 718),
    (BF, DX, T128, False): (20206, 196, 130), (BF, DX, T128, True): (1581, 193, 4858),
    (BF, DX, T256X128, False): (33012, 154, 131), (BF, DX, T256X128, True): (24471, 129, 8854),
    (BF, DX, T256, False): (28488, 408, 130), (BF, DX, T256, True): (6925, 388, 8293),
    (BF, DW, T64, False): (205, 106, 101), (BF, DW, T64, True): (761, 104, 104),
    (BF, DW, T128, False): (164, 8140, 459), (BF, DW, T128, True): (9614, 386, 385),
    (BF, DW_ONE, T64, False): (205, 106, 101), (BF, DW_ONE, T64, True): (761, 104, 104),
    (BF, DW_ONE, T128, False): (164, 8140, 459), (BF, DW_ONE, T128, True): (9614, 386, 385),
    (BF, DW_ONE, T256X128, False): (131, 7211, 1036), (BF, DW_ONE, T256X128, True): (10467, 8338, 130),
    (BF, DW_ONE, T256, False): (132, 1584, 8195), (BF, DW_ONE, T256, True): (89975, 398, 388),
    (BF, DW_TWO, T64, False): (205, 106, 101), (BF, DW_TWO, T64, True): (353, 101, 106),
    (BF, DW_TWO, T128, False): (132, 450, 7088), (BF, DW_TWO, T128, True): (22210, 194, 132),
    (BF, DW_TWO, T256X128, False): (131, 7211, 1036), (BF, DW_TWO, T256X128, True): (37234, 1162, 130),
    (BF, DW_TWO, T256, False): (131, 1546, 7741), (BF, DW_TWO, T256, True): (42110, 388, 388),
}
# (bf16's tiles do not go by residuals)
CASES.update({(BF, FWD_RES, k[2], k[3]): size for k, size in list(CASES.items()) if k[:2] == (BF, FWD)})
KEYS = list(CASES)
IDS = ["%s-%s-%dx%d-%s" % ("bf16" if k[0] == BF else "f32", NAMES[k[1]], *k[2], "split" if k[3] else "whole") for k in KEYS]
# sizes that are whole vectors (no copies) and, the last two, whole tiles
MORE = [(20001, 152, 664), (20001, 664, 152), (40001, 152, 920), (40001, 152, 1304), (600, 1688, 1816), (6001, 216, 856),
        (16384, 256, 512), (8192, 512, 1024)]


def test_the_sizes_reach_every_kernel():
    for key, size in CASES.items():
        dtype, product, tile, split = key
        tm, tn, splits = tiles(cf.dtype_code(dtype), *size, product)
        assert ((tm, tn), splits > 1) == (tile, split), (key, size, tm, tn, splits)
        rows, fin, fout = size
        m, n = {FWD: (rows, fout), FWD_RES: (rows, fout), DX: (rows, fin)}.get(product, (fin, fout))
        assert m > tm and n > tn and m % tm and n % tn
    for dtype in (F32, BF):
        for product in (FWD, FWD_RES, DX, DW, DW_ONE) + ((DW_TWO,) if dtype == BF else ()):
            reached = {(k[2], k[3]) for k in KEYS if k[:2] == (dtype, product)}
            every = [T64, T128] + ([T256X128] if product != DW else []) + ([T256] if product != DW and dtype == BF else [])
            assert reached == {(t, s) for t in every for s in (False, True)}


def test_no_size_takes_another_kernel():
    """The estimate's choices over the range of sizes are those that the cases above cover."""
    sizes = [17, 60, 300, 1000, 4096, 20000, 100000, 400000, 1 << 20]
    widths = [1, 5, 16, 60, 128, 200, 512, 1000, 2048, 4096, 9000, 65536]
    for dtype in (F32, BF):
        for product in (FWD, FWD_RES, DX, DW, DW_ONE, DW_TWO)[:6 if dtype == BF else 5]:
            for rows in sizes:
                for fin in widths:
                    for fout in widths:
                        tm, tn, splits = tiles(cf.dtype_code(dtype), rows, fin, fout, product)
                        assert not tm or (dtype, product, (tm, tn), splits > 1) in CASES


# ------------------------------------------------------------------------- GPU
def made(rows, fin, fout, dtype):
    gen = torch.Generator(device="cuda").manual_seed(rows + 3 * fin + 7 * fout)
    rnd = lambda *shape: torch.randn(*shape, generator=gen, device="cuda")  # noqa: E731
    x, w = (rnd(rows, fin) + 0.25).to(dtype), (rnd(fin, fout) / fin ** 0.5).to(dtype)
    return x, w, rnd(fout), rnd(rows, fout).to(dtype), (1.4 * rnd(rows, fout)).to(dtype), rnd(rows, fout).to(dtype)


def within(got, want, tol):
    if got.dtype == BF:
        tol = tol + 2.0 ** -8 * (want.abs() + tol)
    worst = float(((got.double() - want).abs() / (tol + TINY)).max())
    assert worst <= 1.0, worst


def check_forward(x, w, b, r=None):
    """With pre kept, and without (pre is not an argument of the tiles' choice)."""
    silu = cf.CF_ACT_SILU
    xd, wd, bd = x.double(), w.double(), b.double()
    mag = xd.abs() @ wd.abs()
    z = xd @ wd + bd
    a = z * torch.sigmoid(z)
    ep = (x.shape[1] + 2) * U * mag + U * (z.abs() + bd.abs())
    want = a if r is None else a + r.double()
    ey = 1.1 * ep + U * (8 + 2 * z.abs()) * a.abs() + U * want.abs()
    pre, y = cf.cf_linear_fwd(x, w, b, silu, R=r)
    within(pre, z, ep)
    within(y, want, ey)
    none, served = cf.cf_linear_fwd(x, w, b, silu, R=r, need_pre=False)
    assert none is None and torch.equal(served, y)


def check_backward(x, w, pre, dy, act, slope):
    z, d = pre.double(), dy.double()
    xd, wd, rows, fout = x.double(), w.double(), x.shape[0], w.shape[1]
    if act == cf.CF_ACT_SILU:
        s = torch.sigmoid(z)
        e = U * (16 + 4 * z.abs()) * (1 + z.abs()) * d.abs()
        d = d * (s * (1 + z * torch.sigmoid(-z)))
    else:
        e = torch.zeros_like(d) if slope == 1.0 else U * d.abs()
        d = torch.where(z > 0, d, slope * d)
    if x.dtype == BF and act == cf.CF_ACT_SILU:
        e = e + 2.0 ** -16 * (d.abs() + e)
    dx, dw, db = cf.cf_linear_bwd(x, w, None if slope == 1.0 and act == cf.CF_ACT_LRELU else pre, dy, act, slope)
    wt, xt = wd.t().contiguous(), xd.t().contiguous()
    # (a D in two parts: twice as many products)
    within(dx, d @ wt, e @ wt.abs() + (2 * fout + 2) * U * (d.abs() @ wt.abs()) * 1.01)
    within(dw, xt @ d, xt.abs() @ e + (2 * rows + 2) * U * (xt.abs() @ d.abs()) * 1.01)
    within(db, d.sum(0), e.sum(0) + (rows + 2) * U * d.abs().sum(0))


@pytest.mark.gpu
@pytest.mark.parametrize("key", KEYS, ids=IDS)
def test_kernel(key):
    dtype, product, _, _ = key
    x, w, b, r, pre, dy = made(*CASES[key], dtype)
    if product in (FWD, FWD_RES):
        check_forward(x, w, b, r if product == FWD_RES else None)
    if product in (DX, DW_TWO):
        check_backward(x, w, pre, dy, cf.CF_ACT_SILU, 0.0)
    if product in (DX, DW):
        check_backward(x, w, pre, dy, cf.CF_ACT_LRELU, 1.0)
    if product in (DX, DW_ONE):
        check_backward(x, w, pre, dy, cf.CF_ACT_LRELU, 0.5)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [F32, BF], ids=["f32", "bf16"])
@pytest.mark.parametrize("size", MORE, ids=str)
def test_rows_of_whole_vectors(size, dtype):
    x, w, b, r, pre, dy = made(*size, dtype)
    check_forward(x, w, b)
    check_forward(x, w, b, r)
    check_backward(x, w, pre, dy, cf.CF_ACT_SILU, 0.0)
    check_backward(x, w, pre, dy, cf.CF_ACT_LRELU, 1.0)
