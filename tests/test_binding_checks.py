"""What the bindings of group norm, Newton-Schulz and Muon refuse before a
kernel is launched (host tensors are enough: nothing here reaches the GPU)."""
import pytest
import torch

from cnn_cosmology_volumes_amd import cf

BF = torch.bfloat16


def _gn(**kw):
    x, v = torch.zeros(2, 4, 4, 4, 8), torch.zeros(8)
    return cf.cf_groupnorm_fwd(x, 2, v, v, 1e-5, **kw)


def _gn_bwd(**kw):
    x, v, m = torch.zeros(2, 4, 4, 4, 8), torch.zeros(8), torch.zeros(2, 2)
    return cf.cf_groupnorm_bwd(x, x, 2, v, v, m, m, **kw)


OUTPUTS = [("Y", torch.zeros(2, 4, 4, 4, 8, dtype=BF), TypeError),            # half of what is written
           ("Y", torch.zeros(1, 4, 4, 4, 8), ValueError),
           ("Y", torch.zeros(8, 4, 4, 4, 2).transpose(0, 4), ValueError),      # strides
           ("mean", torch.zeros(2, 1), ValueError),
           ("mean", torch.zeros(2, 2, dtype=torch.float64), TypeError),
           ("rstd", torch.zeros(2), ValueError),
           ("rstd", torch.zeros(2, 4)[:, ::2], ValueError)]


@pytest.mark.parametrize("name,t,error", OUTPUTS, ids=["%s-%d" % (o[0], i) for i, o in enumerate(OUTPUTS)])
def test_groupnorm_outputs(name, t, error):
    with pytest.raises(error, match=name):
        _gn(**{name: t})


@pytest.mark.parametrize("t,error", [(torch.zeros(2, 4, 4, 4, 8, dtype=BF), TypeError),
                                     (torch.zeros(2, 4, 4, 4, 4), ValueError),
                                     (torch.zeros(2, 4, 4, 4, 16)[..., ::2], ValueError)])
def test_groupnorm_backward_output(t, error):
    with pytest.raises(error, match="dX"):
        _gn_bwd(dX=t)


@pytest.mark.parametrize("call", [_gn, _gn_bwd])
def test_workspace_with_gaps(call):
    with pytest.raises(ValueError, match="ws"):
        call(ws=torch.zeros(1 << 16, dtype=torch.uint8)[::2])


def test_matrix_workspace_with_gaps():
    ws = torch.zeros(1 << 22, dtype=torch.uint8)[::2]
    x = torch.zeros(4, 6)
    with pytest.raises(ValueError, match="ws"):
        cf.cf_newton_schulz(cf.newton_schulz_params(), [x], ws=ws)
    with pytest.raises(ValueError, match="ws"):
        cf.cf_muon(cf.muon_params(0.1), [x], [x.clone()], [x.clone()], ws=ws)


def _host_calls():
    x, v, m, w = torch.zeros(2, 4, 4, 4, 8), torch.zeros(8), torch.zeros(2, 2), torch.zeros(4, 6)
    ns, hp = cf.newton_schulz_params(), cf.muon_params(0.1)
    return {"groupnorm_fwd": lambda: cf.cf_groupnorm_fwd(x, 2, v, v, 1e-5),
            "groupnorm_bwd": lambda: cf.cf_groupnorm_bwd(x, x, 2, v, v, m, m),
            "newton_schulz": lambda: cf.cf_newton_schulz(ns, [w]),
            "muon": lambda: cf.cf_muon(hp, [w], [w.clone()], [w.clone()])}


@pytest.mark.parametrize("name", sorted(_host_calls()))
def test_host_tensors(name):
    """A host address must not reach a kernel."""
    with pytest.raises(ValueError, match="GPU"):
        _host_calls()[name]()


@pytest.mark.parametrize("where", ["x", "dy", "gamma", "beta", "mean", "rstd", "Y", "dX", "ws"])
def test_one_tensor_elsewhere(where):
    """Each argument is looked at, not the first one alone.  (A stand-in for
    the GPU's index lets the checks run on any machine.)"""
    class Here(torch.Tensor):
        def get_device(self):
            return 0

    def t(name, *shape, dtype=torch.float32):
        a = torch.zeros(*shape, dtype=dtype)
        return a if name == where else a.as_subclass(Here)

    x, dy, gamma, beta = t("x", 2, 4, 4, 4, 8), t("dy", 2, 4, 4, 4, 8), t("gamma", 8), t("beta", 8)
    mean, rstd = t("mean", 2, 2), t("rstd", 2, 2)
    out, ws = t("Y", 2, 4, 4, 4, 8), t("ws", 1 << 16, dtype=torch.uint8)
    dx = t("dX", 2, 4, 4, 4, 8)
    if where not in ("dy", "dX"):
        with pytest.raises(ValueError, match="GPU"):
            cf.cf_groupnorm_fwd(x, 2, gamma, beta, 1e-5, Y=out, mean=mean, rstd=rstd, ws=ws)
    if where != "Y":
        with pytest.raises(ValueError, match="GPU"):
            cf.cf_groupnorm_bwd(x, dy, 2, gamma, beta, mean, rstd, dX=dx, ws=ws)


@pytest.mark.parametrize("where", ["matrix", "output", "param", "gradient", "momentum", "ws"])
def test_one_matrix_elsewhere(where):
    class Here(torch.Tensor):
        def get_device(self):
            return 0

    def t(name, *shape, dtype=torch.float32):
        a = torch.zeros(*shape, dtype=dtype)
        return a if name == where else a.as_subclass(Here)

    ws = t("ws", 1 << 22, dtype=torch.uint8)
    if where in ("matrix", "output", "ws"):
        with pytest.raises(ValueError, match="GPU"):
            cf.cf_newton_schulz(cf.newton_schulz_params(), [t("", 4, 6), t("matrix", 4, 6)],
                                out=[t("", 4, 6), t("output", 4, 6)], ws=ws)
    if where in ("param", "gradient", "momentum", "ws"):
        with pytest.raises(ValueError, match="GPU"):
            cf.cf_muon(cf.muon_params(0.1), [t("", 4, 6), t("param", 4, 6)], [t("", 4, 6), t("gradient", 4, 6)],
                       [t("", 4, 6), t("momentum", 4, 6)], ws=ws)
