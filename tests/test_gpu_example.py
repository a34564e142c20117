"""Group norm and Muon together, as the example trains with them."""
import os
import sys

import pytest
import torch

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
import groupnorm_muon as ex  # noqa: E402
from cnn_cosmology_volumes_amd import cf  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_training_lowers_the_loss(dtype):
    """Twelve steps on one batch of four: enough capacity to fit it, so the
    last loss is well below the first."""
    losses = ex.main(["--size", "16", "--steps", "12", "--dtype", dtype])
    assert losses[-1] < 0.5 * losses[0]


@pytest.mark.parametrize("name", ["conv", "gamma", "beta", "dense", "bias"])
def test_gradients_against_differences(name):
    """The directional derivative of the fp32 loss along random directions of
    one kind of parameter, with a linear head (the loss is smooth then).  The
    difference quotient with step h / 2 is off by a third of the change from h
    to h / 2 and higher powers of h, and by the fp32 rounding of the two
    losses, 2^-18 of the loss each (the sums of a layer of up to 864 terms, and
    five layers), over h."""
    x, t = ex.batch(16, 3, torch.float32, seed=5)
    net = ex.Net(16, dtype=torch.float32, seed=6)
    net.slope = 1.0
    params = getattr(net, name)
    loss, saved = net.forward(x, t)
    grads = net.backward(saved)[name]
    gen = torch.Generator(device="cuda").manual_seed(1)
    for trial in range(3):
        v = [torch.randn(p.shape, generator=gen, device="cuda") * p.abs().mean().clamp(min=0.05) for p in params]
        want = sum((g.double() * d.double()).sum() for g, d in zip(grads, v)).item()

        def quotient(h):
            ends = []
            for s in (h, -h):
                setattr(net, name, [p + s * d for p, d in zip(params, v)])
                ends.append(net.forward(x, t)[0].item())
            setattr(net, name, params)
            return (ends[0] - ends[1]) / (2 * h)

        h = 2.0 ** -6
        wide, near = quotient(h), quotient(h / 2)
        tol = 2 * abs(wide - near) + 2.0 ** -18 * loss.item() / (h / 2)
        assert abs(near - want) <= tol, (trial, near, want, tol)


def test_momenta_and_weights_follow_muon():
    """A step changes the matrices by Muon's update of their gradients and the
    vectors by SGD's."""
    x, t = ex.batch(16, 2, torch.float32, seed=7)
    net = ex.Net(16, dtype=torch.float32, seed=8)
    hp = cf.muon_params(0.02)
    mats = [w.clone() for w in net.conv + net.dense]
    vecs = [p.clone() for p in net.gamma + net.beta + net.bias]
    g = net.backward(net.forward(x, t)[1])
    net.step(x, t, hp, 0.1)
    m = [torch.zeros_like(w) for w in mats]
    cf.cf_muon(hp, mats, g["conv"] + g["dense"], m)
    for a, b in zip(mats + m, net.conv + net.dense + net.momenta):
        assert torch.equal(a, b)
    for p, d, q in zip(vecs, g["gamma"] + g["beta"] + g["bias"], net.gamma + net.beta + net.bias):
        assert torch.allclose(p - 0.1 * d, q, rtol=0, atol=2.0 ** -23 * float(p.abs().max() + 0.1 * d.abs().max()))
