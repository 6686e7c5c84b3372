"""Layer norm of rows whose elements are all equal: the mean is that element, the
deviations are zero and the output is beta, at every width."""
from __future__ import annotations

import pytest
import torch

import test_layer_norm_gpu as ln

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda:0")


@pytest.fixture(scope="module")
def g():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    from dense_fp16_gemm_05_gb300 import build as gbuild
    gbuild.build()
    from dense_fp16_gemm_05_gb300 import gemm_f16
    gemm_f16.lib()
    return gemm_f16


# 57600 = 225 * 2^8 and 56.25 = 225 * 2^-2 have eight significant bits, so sums of up
# to 2^16 of them are exact in fp32 in any order, and so is their division by the
# number of them.  In these widths the sum times the rounded 1 / dim is not 57600.
@pytest.mark.parametrize("value", [57600.0, -56.25])
@pytest.mark.parametrize("xt,wt", ln.TYPES)
@pytest.mark.parametrize("dim", [7, 14, 56, 104, 448, 896, 1000, 1663, 1664, 3584, 5248, 6080, 9519, 9524, 19040])
def test_output_is_beta(g, dim, xt, wt, value):
    x = torch.full((5, dim), value, dtype=ln.DTYPES[xt], device=DEV)
    _, _, w, b = ln.draw(1, dim, ln.DTYPES[xt], ln.DTYPES[wt], dim)
    Y, mean, rstd = g.layer_norm_fwd(x, w, b, eps=ln.EPS)
    assert (mean == value).all()
    assert torch.equal(Y, b.to(x.dtype).expand_as(Y))
    # eps in fp32, its root, its reciprocal: a rounding each
    assert ((rstd.double() - ln.EPS ** -0.5).abs() <= 4 * ln.U * ln.EPS ** -0.5).all()
