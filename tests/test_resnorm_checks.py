"""cf_resnorm_fwd / _bwd's checks of sizes, in the binding and in the library (no GPU needed)."""
import pytest
import torch

from cnn_cosmology_volumes_amd import cf


@pytest.mark.parametrize("shape", [(1, 1, 1, (1 << 30) + 1, 1), ((1 << 30) + 1, 1, 1, 1, 1), (4, 8), (2, 2, 2, 8)], ids=str)
def test_the_binding_says_what_it_takes(shape):
    """Five dimensions, each of 2^30 at most, which is the library's own limit: cf_dims holds 64 bits, so nothing wraps."""
    x = torch.empty(shape, dtype=torch.bfloat16, device="meta")
    for call in (lambda: cf.cf_resnorm_fwd(x, x, cf.CF_NORM_RMS, 1e-6), lambda: cf.cf_resnorm_bwd(x, x, x, x, cf.CF_NORM_RMS, 1e-6)):
        with pytest.raises(ValueError, match=r"NDHWC tensors, 2\^30 at most along a dimension"):
            call()


def test_the_librarys_limits():
    size = lambda *shape: cf.cf_resnorm_workspace_size(cf.CF_F32, shape, 0)  # noqa: E731
    assert size(1, 1, 1, 1 << 30, 1) > 0
    assert size(1, 1, 1, (1 << 30) + 1, 1) == 0 and b"too large" in cf.lib().cf_last_error()
    assert size(1, 1, 1, (1 << 32) + 8, 1) == 0
    assert size(1 << 20, 1 << 11, 1 << 10, 1, 1) == 0 and size(1, 1, 1, 1, 4097) == 0
