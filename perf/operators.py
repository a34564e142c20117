"""Cases of the group-norm and Muon operators: inputs, plain forms, exact
values and the work each pass cannot do without.

Operators
---------
gn_fwd   group norm + activation of an NDHWC tensor -> y, mean, rstd
gn_bwd   its backward from the saved mean and rstd -> dx, dgamma, dbeta
ns       Newton-Schulz orthogonalisation of one matrix (5 quintic steps)
muon     Muon's update of a list of weight matrices -> weights, momenta

`own = False` computes them with elementary torch operations, `own = True`
calls libcf's entry points through its Python binding.
"""
import math

import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
EPS = 1e-5                           # group norm
NS_A, NS_B, NS_C = 3.4445, -4.7750, 2.0315
NS_STEPS, NS_EPS = 5, 1e-7
LR, MU, WD = 0.02, 0.95, 0.01

# conv weights [27 cin, cout] and dense weights [in, out] of the 128^3
# benchmark network, and of the extended network with 7 conv layers
BLOCK_NET = "108x32,864x64,1728x128,3456x256,6912x256,16384x128,128x64,64x3"
TABLE1_NET = "108x16,432x32,864x64,1728x128,3456x256,6912x256,6912x256,2048x2048,2048x256,256x4"


def listed():
    return [
        # the smallest call: a deep layer's 4^3 volume, one sample
        {"name": "gn_fwd_4c256_b1", "op": "gn_fwd", "n": 1, "d": 4, "h": 4, "w": 4, "c": 256, "groups": 32,
         "dtype": "bf16", "act": "silu", "slope": 1.0},
        # first block's conv output of the 128^3 network, batch 8 (1.07 GB)
        {"name": "gn_fwd_128c32_b8", "op": "gn_fwd", "n": 8, "d": 128, "h": 128, "w": 128, "c": 32, "groups": 8,
         "dtype": "bf16", "act": "lrelu", "slope": 0.3},
        # an odd volume with 5 channels a group, fp32
        {"name": "gn_fwd_ragged_f32", "op": "gn_fwd", "n": 3, "d": 37, "h": 29, "w": 31, "c": 60, "groups": 12,
         "dtype": "f32", "act": "silu", "slope": 1.0},
        # a small fp32 layer's backward
        {"name": "gn_bwd_8c256_b2_f32", "op": "gn_bwd", "n": 2, "d": 8, "h": 8, "w": 8, "c": 256, "groups": 32,
         "dtype": "f32", "act": "lrelu", "slope": 0.3},
        # second block's conv output, batch 8
        {"name": "gn_bwd_64c64_b8", "op": "gn_bwd", "n": 8, "d": 64, "h": 64, "w": 64, "c": 64, "groups": 16,
         "dtype": "bf16", "act": "lrelu", "slope": 0.3},
        # an odd volume, groups of 12 channels, bf16
        {"name": "gn_bwd_ragged_bf16", "op": "gn_bwd", "n": 2, "d": 45, "h": 33, "w": 27, "c": 96, "groups": 8,
         "dtype": "bf16", "act": "silu", "slope": 1.0},
        # first conv layer's weight gradient: the smallest matrix
        {"name": "ns_108x32", "op": "ns", "rows": 108, "cols": 32, "dtype": "f32"},
        # odd sizes, wide rather than tall
        {"name": "ns_333x1001", "op": "ns", "rows": 333, "cols": 1001, "dtype": "f32"},
        # a square bf16 matrix
        {"name": "ns_2048x2048_bf16", "op": "ns", "rows": 2048, "cols": 2048, "dtype": "bf16"},
        # the largest matrix
        {"name": "ns_4096x4096", "op": "ns", "rows": 4096, "cols": 4096, "dtype": "f32"},
        # one optimizer step over the matrices of each network
        {"name": "muon_block_net", "op": "muon", "shapes": BLOCK_NET, "nesterov": True, "scale": "aspect"},
        {"name": "muon_table1_net", "op": "muon", "shapes": TABLE1_NET, "nesterov": False, "scale": "rms"},
    ]


def _log_int(rng, lo, hi):
    return min(hi, int(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))


def draw(rng):
    op = rng.choice(["gn_fwd", "gn_bwd", "ns", "muon"])
    if op in ("gn_fwd", "gn_bwd"):
        groups = rng.choice([1, 2, 3, 4, 6, 8, 12, 16, 32])
        c = groups * _log_int(rng, 1, 24)
        n = rng.choice([1, 1, 2, 3, 4, 8])
        size = [_log_int(rng, 1, 72) for _ in range(3)]
        while n * c * size[0] * size[1] * size[2] > 1 << 26:
            size[size.index(max(size))] //= 2
        if size[0] * size[1] * size[2] * c < 8 * groups:
            c = 8 * groups               # a group of one or two values has a gradient of rounding errors only
        return {"op": op, "n": n, "d": size[0], "h": size[1], "w": size[2], "c": c, "groups": groups,
                "dtype": rng.choice(["f32", "bf16"]), "act": rng.choice(["lrelu", "silu"]),
                "slope": rng.choice([0.0, 0.1, 0.3, 1.0])}
    if op == "ns":
        rows, cols = _log_int(rng, 1, 4096), _log_int(rng, 1, 2048)
        if rng.random() < 0.3:
            rows, cols = cols, rows
        return {"op": op, "rows": rows, "cols": cols, "dtype": rng.choice(["f32", "bf16"])}
    shapes = ["%dx%d" % (_log_int(rng, 1, 4096), _log_int(rng, 1, 512)) for _ in range(rng.randint(1, 8))]
    return {"op": op, "shapes": ",".join(shapes), "nesterov": rng.random() < 0.5,
            "scale": rng.choice(["aspect", "rms"])}


def _shapes(case):
    return [tuple(int(v) for v in s.split("x")) for s in case["shapes"].split(",")]


# ------------------------------------------------------------------- inputs
def _gradient(gen, rows, cols):
    """A weight gradient: a few strong directions over a noise floor."""
    r = min(4, rows, cols)
    u = torch.randn(rows, r, generator=gen, device="cuda")
    v = torch.randn(r, cols, generator=gen, device="cuda")
    s = 0.6 ** torch.arange(r, device="cuda", dtype=torch.float32)
    low = (u[:, :, None] * (s[:, None] * v)[None]).sum(1) if rows * cols <= 1 << 16 else (u * s) @ v
    return 1e-3 * (low + torch.randn(rows, cols, generator=gen, device="cuda"))


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    st = {"case": case}
    if case["op"] in ("gn_fwd", "gn_bwd"):
        n, c, g, dt = case["n"], case["c"], case["groups"], DTYPES[case["dtype"]]
        shape = (n, case["d"], case["h"], case["w"], c)
        # conv outputs: each channel with an offset and a spread of its own
        x = torch.randn(shape, generator=gen, device="cuda")
        x.mul_(0.5 + torch.rand(c, generator=gen, device="cuda"))
        x.add_(torch.randn(c, generator=gen, device="cuda"))
        st["x"] = x.to(dt)
        st["gamma"] = 0.5 + torch.rand(c, generator=gen, device="cuda")
        st["beta"] = torch.rand(c, generator=gen, device="cuda") - 0.5
        if case["op"] == "gn_bwd":
            st["dy"] = torch.randn(shape, generator=gen, device="cuda").to(dt)
            # what the forward pass left
            t = st["x"].reshape(n, -1, g, c // g)
            mean = t.sum((1, 3), dtype=torch.float64) / (t.shape[1] * t.shape[3])
            t = t.float() - mean.float()[:, None, :, None]
            var = t.square().sum((1, 3), dtype=torch.float64) / (t.shape[1] * t.shape[3])
            st["mean"], st["rstd"] = mean.float(), (var + EPS).rsqrt().float()
    elif case["op"] == "ns":
        st["x"] = _gradient(gen, case["rows"], case["cols"]).to(DTYPES[case["dtype"]])
    else:
        st["w"], st["g"], st["m"] = [], [], []
        for rows, cols in _shapes(case):
            st["w"].append(torch.randn(rows, cols, generator=gen, device="cuda") * math.sqrt(2.0 / rows))
            st["g"].append(_gradient(gen, rows, cols))
            st["m"].append(4 * _gradient(gen, rows, cols))
    return st


# -------------------------------------------------------------- plain forms
def _plain_gn_fwd(st):
    case, x = st["case"], st["x"]
    n, c, g = case["n"], case["c"], case["groups"]
    t = x.float().reshape(n, -1, g, c // g)
    count = t.shape[1] * t.shape[3]
    mean = (t.sum((1, 3), dtype=torch.float64) / count).float()
    t = t - mean[:, None, :, None]
    rstd = ((t * t).sum((1, 3), dtype=torch.float64) / count + EPS).rsqrt().float()
    z = t * rstd[:, None, :, None] * st["gamma"].reshape(g, -1) + st["beta"].reshape(g, -1)
    if case["act"] == "silu":
        y = z / (1 + torch.exp(-z))
    else:
        y = torch.where(z > 0, z, case["slope"] * z)
    return y.to(x.dtype).reshape(x.shape), mean, rstd


def _plain_gn_bwd(st):
    case, x = st["case"], st["x"]
    n, c, g = case["n"], case["c"], case["groups"]
    shape = (n, -1, g, c // g)
    gamma, beta = st["gamma"].reshape(g, -1), st["beta"].reshape(g, -1)
    mean, rstd = st["mean"][:, None, :, None], st["rstd"][:, None, :, None]
    xhat = (x.float().reshape(shape) - mean) * rstd
    dz = st["dy"].float().reshape(shape)
    if case["act"] == "silu":
        z = xhat * gamma + beta
        s = 1 / (1 + torch.exp(-z))
        dz = dz * (s * (1 + z * (1 - s)))
    else:
        # the derivative jumps at z = 0: its sign is taken in 64 bits
        z = (x.reshape(shape).double() - mean.double()) * rstd.double() * gamma.double() + beta.double()
        dz = torch.where(z > 0, dz, case["slope"] * dz)
    a = dz.sum(1, dtype=torch.float64)
    b = (dz * xhat).sum(1, dtype=torch.float64)
    count = xhat.shape[1] * xhat.shape[3]
    s1 = ((gamma * a).sum(-1) / count).float()[:, None, :, None]
    s2 = ((gamma * b).sum(-1) / count).float()[:, None, :, None]
    dx = rstd * (gamma * dz - s1 - xhat * s2)
    return dx.to(x.dtype).reshape(x.shape), b.sum(0).float().reshape(c), a.sum(0).float().reshape(c)


def _plain_ns(x):
    y = x.float()
    if y.shape[0] > y.shape[1]:
        y = y.t()
    y = y / (y.double().square().sum().sqrt().float() + NS_EPS)
    for _ in range(NS_STEPS):
        a = y @ y.t()
        y = NS_A * y + (NS_B * a + NS_C * (a @ a)) @ y
    return y.t() if x.shape[0] > x.shape[1] else y


def _factor(case, rows, cols):
    return math.sqrt(max(1.0, cols / rows)) if case["scale"] == "aspect" else 0.2 * math.sqrt(max(rows, cols))


def _plain_muon(st):
    case = st["case"]
    for w, g, m in zip(st["w"], st["g"], st["m"]):
        m.mul_(MU).add_(g)
        u = g + MU * m if case["nesterov"] else m
        w.mul_(1 - LR * WD).sub_((LR * _factor(case, *w.shape)) * _plain_ns(u))
    return st["w"], st["m"]


# -------------------------------------------------------------------- calls
def _own(st):
    from cnn_cosmology_volumes_amd import cf
    case = st["case"]
    if case["op"] in ("gn_fwd", "gn_bwd"):
        act = cf.CF_ACT_SILU if case["act"] == "silu" else cf.CF_ACT_LRELU
        if case["op"] == "gn_fwd":
            return cf.cf_groupnorm_fwd(st["x"], case["groups"], st["gamma"], st["beta"], EPS, act, case["slope"])
        return cf.cf_groupnorm_bwd(st["x"], st["dy"], case["groups"], st["gamma"], st["beta"], st["mean"],
                                   st["rstd"], act, case["slope"])
    ns = cf.newton_schulz_params(NS_STEPS, NS_A, NS_B, NS_C, NS_EPS)
    if case["op"] == "ns":
        return cf.cf_newton_schulz(ns, [st["x"]])[0]
    scale = cf.CF_MUON_SCALE_ASPECT if case["scale"] == "aspect" else cf.CF_MUON_SCALE_RMS
    hp = cf.muon_params(LR, momentum=MU, nesterov=case["nesterov"], weight_decay=WD, scale=scale, ns=ns)
    cf.cf_muon(hp, st["w"], st["g"], st["m"])
    return st["w"], st["m"]


def run(st):
    if own:
        return _own(st)
    op = st["case"]["op"]
    if op == "gn_fwd":
        return _plain_gn_fwd(st)
    if op == "gn_bwd":
        return _plain_gn_bwd(st)
    if op == "ns":
        return _plain_ns(st["x"]).to(st["x"].dtype).contiguous()
    return _plain_muon(st)


# --------------------------------------------------------------------- work
def _ns_flops(rows, cols):
    # per step: A = X X^T and A^2 are symmetric (half of each product), then B X
    m, n = min(rows, cols), max(rows, cols)
    return NS_STEPS * (m * m * n + m * m * m + 2 * m * m * n)


def work(case):
    if case["op"] in ("gn_fwd", "gn_bwd"):
        e = case["n"] * case["d"] * case["h"] * case["w"] * case["c"]
        size = 4 if case["dtype"] == "f32" else 2
        stats = 2 * case["n"] * case["groups"] * 4
        if case["op"] == "gn_fwd":
            return {"bytes": 2 * e * size + 8 * case["c"] + stats, "flops": 8 * e}
        return {"bytes": 3 * e * size + 16 * case["c"] + stats, "flops": 16 * e}
    if case["op"] == "ns":
        size = 4 if case["dtype"] == "f32" else 2
        return {"bytes": 2 * case["rows"] * case["cols"] * size, "flops": _ns_flops(case["rows"], case["cols"])}
    shapes = _shapes(case)
    return {"bytes": sum(20 * r * c for r, c in shapes), "flops": sum(_ns_flops(r, c) + 6 * r * c for r, c in shapes)}


# -------------------------------------------------------------------- exact
def _exact_gn(st):
    """From the definition, one sample and group at a time, in 64 bits."""
    case = st["case"]
    n, c, g = case["n"], case["c"], case["groups"]
    x = st["x"].reshape(n, -1, c)
    cg = c // g
    first = torch.empty(x.shape, dtype=torch.float64, device="cuda")
    second = torch.zeros(n, c, dtype=torch.float64, device="cuda")
    third = torch.zeros(n, c, dtype=torch.float64, device="cuda")
    means, rstds = [], []
    for i in range(n):
        for j in range(g):
            ch = slice(j * cg, (j + 1) * cg)
            v = x[i, :, ch].double()
            gamma, beta = st["gamma"][ch].double(), st["beta"][ch].double()
            if case["op"] == "gn_fwd":
                var, mu = torch.var_mean(v, correction=0)
                r = 1.0 / torch.sqrt(var + EPS)
                means.append(mu)
                rstds.append(r)
            else:
                mu, r = st["mean"][i, j].double(), st["rstd"][i, j].double()
            h = (v - mu) * r
            z = torch.addcmul(beta, h, gamma)
            if case["op"] == "gn_fwd":
                if case["act"] == "silu":
                    first[i, :, ch] = z * torch.sigmoid(z)
                else:
                    first[i, :, ch] = z.clamp(min=0) + case["slope"] * z.clamp(max=0)
                continue
            if case["act"] == "silu":
                q = torch.sigmoid(z)
                slope = q + z * q * torch.sigmoid(-z)
            else:
                slope = case["slope"] + (1 - case["slope"]) * (z > 0).double()
            t = st["dy"].reshape(n, -1, c)[i, :, ch].double() * slope
            second[i, ch] = (t * h).sum(0)
            third[i, ch] = t.sum(0)
            t = t * gamma
            first[i, :, ch] = (t - t.mean() - h * (t * h).mean()) * r
    first = first.reshape(st["x"].shape)
    if case["op"] == "gn_fwd":
        return first, torch.stack(means).reshape(n, g), torch.stack(rstds).reshape(n, g)
    return first, second.sum(0), third.sum(0)


def _exact_ns(x):
    """The quintic step with the long side in rows: X (a + b G + c G^2)."""
    t = x.double()
    wide = t.shape[1] > t.shape[0]
    if wide:
        t = t.t().contiguous()
    t = t / (torch.linalg.vector_norm(t) + NS_EPS)
    eye = torch.eye(t.shape[1], dtype=torch.float64, device="cuda")
    for _ in range(NS_STEPS):
        g = t.t() @ t
        t = t @ (NS_A * eye + g @ (NS_B * eye + NS_C * g))
    return t.t() if wide else t


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] in ("gn_fwd", "gn_bwd"):
        return _exact_gn(st)
    if case["op"] == "ns":
        return _exact_ns(st["x"]).contiguous()
    ws, ms = [], []
    for w, g, m in zip(st["w"], st["g"], st["m"]):
        g, m = g.double(), m.double()
        m = m * MU + g
        o = _exact_ns(g + m * MU if case["nesterov"] else m)
        ws.append(w.double() - LR * (WD * w.double() + _factor(case, *w.shape) * o))
        ms.append(m)
    return ws, ms
