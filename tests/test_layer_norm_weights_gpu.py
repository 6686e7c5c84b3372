"""Layer norm with weights that lie off the grid of X's pieces: a slice of a flat
parameter buffer beside rows that are aligned, in every kernel's range of widths."""
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


def moved(t, by):
    """t `by` elements into an allocation of its own."""
    flat = torch.empty(t.numel() + by, dtype=t.dtype, device=DEV)
    flat[by:].copy_(t.reshape(-1))
    return flat[by:].reshape(t.shape)


# Widths of the lane, warp, register and ring kernels, of pieces of 16 and of 4
# bytes, and of rows longer than a block.
@pytest.mark.parametrize("dim", [2, 40, 258, 514, 1030, 2048, 4096, 4100, 6002, 10002, 16384, 16386])
@pytest.mark.parametrize("wt", ["16", "32"])
@pytest.mark.parametrize("xt", ["fp16", "bf16"])
def test_weights_one_element_into_their_allocation(g, dim, wt, xt):
    t = ln.DTYPES[xt]
    x, dy, w, b = ln.draw(5, dim, t, torch.float32 if wt == "32" else t, dim)
    for by in (1, 2, 3):
        for gamma, beta in ((moved(w, by), b), (w, moved(b, by)), (moved(w, by), moved(b, by))):
            mean, rstd = ln.check_forward(g, x, gamma, beta)
        ln.check_backward(g, x, dy, moved(w, by), mean, rstd, w.dtype)
    # rows two elements in: four-byte pieces, whatever the width
    mean, rstd = ln.check_forward(g, moved(x, 2), moved(w, 1), moved(b, 1))
    ln.check_backward(g, moved(x, 2), moved(dy, 2), moved(w, 1), mean, rstd, w.dtype)


@pytest.mark.parametrize("dim", [40, 1028, 4096])
def test_fp32_rows_and_weights_off_the_grid(g, dim):
    x, dy, w, b = ln.draw(5, dim, torch.float32, torch.float32, dim)
    for by in (1, 2):
        mean, rstd = ln.check_forward(g, x, moved(w, by), moved(b, by))
        ln.check_backward(g, x, dy, moved(w, by), mean, rstd, torch.float32)
