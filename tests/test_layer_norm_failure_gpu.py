"""The bounded wait of the layer norm's backward ring, made to run out without a
fault: no row is loaded, every block leaves at its first row's barrier."""
from __future__ import annotations

import pytest
import torch

import test_layer_norm_gpu as ln

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda:0")
SITE_NORM_ROW = 9


@pytest.fixture(scope="module")
def g():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    from dense_fp16_gemm_05_gb300 import build as gbuild
    gbuild.build()
    from dense_fp16_gemm_05_gb300 import gemm_f16
    gemm_f16.lib()
    return gemm_f16


# Full and partly filled blocks, 8 and 16 elements per thread, rows read twice from
# the ring (16384 fp16), rows off the 16-byte grid, fewer and more rows than blocks.
@pytest.mark.parametrize("xt,rows,dim", [("fp16", 3, 1024), ("fp16", 700, 4096), ("bf16", 400, 5000), ("fp16", 40, 16384),
                                         ("fp32", 400, 2047), ("fp16", 400, 4100), ("fp32", 7, 8192)])
def test_wait_runs_out_and_context_survives(g, xt, rows, dim):
    x, dy, w, b = ln.draw(rows, dim, ln.DTYPES[xt], ln.DTYPES[xt], dim)
    _, mean, rstd = g.layer_norm_fwd(x, w, b, eps=ln.EPS)
    dX = torch.full_like(x, 5.0)
    assert g.check() == g.GEMM_OK
    st = g.lib().layer_norm_bwd_selftest_timeout(dy.data_ptr(), x.data_ptr(), mean.data_ptr(), rstd.data_ptr(),
                                                 dX.data_ptr(), rows, dim, g.TYPES[x.dtype], 1 << 20,
                                                 torch.cuda.current_stream().cuda_stream)
    assert st == g.GEMM_OK
    assert g.check() == g.GEMM_ERR_TIMEOUT
    assert (g.last_timeout_record() & 0xFF) == SITE_NORM_ROW, hex(g.last_timeout_record())
    assert (dX == 5.0).all()
    ln.check_backward(g, x, dy, w, mean, rstd, w.dtype)
