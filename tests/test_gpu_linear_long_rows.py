"""Linear layers of few rows with long or wide weights, on both sides of the rules for one launch,
against the fp64 oracle; tolerances of test_gpu_linear.py."""
import pytest

from test_gpu_linear import BF, F32, both

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [F32, BF], ids=["f32", "bf16"])
@pytest.mark.parametrize("fin,fout", [(65536, 24), (16384, 1024), (16384, 515), (8192, 2047), (4097, 512), (8200, 64)])
@pytest.mark.parametrize("rows", [1, 4, 5, 16])
def test_matches_oracle(rows, fin, fout, dtype):
    both(rows, fin, fout, dtype, "silu", 0.0)
    both(rows, fin, fout, dtype, "lrelu", 1.0, bias=False, residual=False, seed=1)


@pytest.mark.parametrize("dtype", [F32, BF], ids=["f32", "bf16"])
@pytest.mark.parametrize("fin,fout", [(16, 16384), (15, 65535), (1024, 4096), (1023, 4097), (16385, 17), (65536, 16), (2048, 2048),
                                      (2047, 1025), (4096, 512)])
@pytest.mark.parametrize("rows", [1, 8, 9, 16])
def test_wide_and_tall(rows, fin, fout, dtype):
    both(rows, fin, fout, dtype, "silu", 0.0)
    both(rows, fin, fout, dtype, "lrelu", 1.0, bias=False, residual=False, seed=1)
