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
