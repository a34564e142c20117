"""cf_grad_clip's checks of its lists: one rule for every tensor, whatever else is in the list."""
import ctypes

import pytest
import torch

from cnn_cosmology_volumes_amd import cf


@pytest.mark.parametrize("others", [[], [torch.zeros(4)], [torch.zeros(4, dtype=torch.bfloat16)]], ids=["alone", "fine", "type"])
@pytest.mark.parametrize("grad,out", [((2, 3), (6,)), ((6,), (2, 3)), ((2, 3), (3, 2)), ((1,), ()), ((5,), (6,))], ids=str)
def test_an_outputs_shape_is_its_gradients(grad, out, others):
    """An output of as many values but another shape is refused, beside tensors of a wrong type or alone."""
    g, o = [torch.zeros(grad), *others], [torch.zeros(out), *others]
    with pytest.raises(ValueError, match="output 0 must have shape"):
        cf.cf_grad_clip(g, 1.0, out=o)
    if not others:
        with pytest.raises(ValueError, match="output 1 must have shape"):
            cf.cf_grad_clip([torch.zeros(4), *g], 1.0, out=[torch.zeros(4), *o])


def test_the_first_that_is_wrong_is_named():
    g = [torch.zeros(2, 3), torch.zeros(4)]
    with pytest.raises(TypeError, match="output 1"):
        cf.cf_grad_clip(g, 1.0, out=[torch.zeros(2, 3), torch.zeros(4, dtype=torch.bfloat16)])
    with pytest.raises(ValueError, match="output 0 must be contiguous"):
        cf.cf_grad_clip(g, 1.0, out=[torch.zeros(3, 2).t(), torch.zeros(4)])
    with pytest.raises(ValueError, match="GPU"):
        cf.cf_grad_clip(g, 1.0, out=[torch.zeros(2, 3), torch.zeros(4)])


def test_lists_that_are_too_large_together():
    """128 tensors of 2^36 values are each allowed, but their chunks together are 2^31."""
    size = lambda count: cf.lib().cf_grad_clip_workspace_size(cf.CF_F32, count, (ctypes.c_int64 * 128)(*[1 << 36] * 128))  # noqa: E731
    assert size(16) > 0 and size(17) == 0 and size(128) == 0
    assert b"too large" in cf.lib().cf_last_error()
