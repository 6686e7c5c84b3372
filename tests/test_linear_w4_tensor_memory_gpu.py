"""GPU tests of the tensor memory kernel of products with 4-bit weights: waits that run
out, streams and replays, and what lies beside X."""
from __future__ import annotations

import pytest
import torch

from test_linear_w4_gpu import DEV, DTYPES, check, g, packed  # noqa: F401  (g: a fixture)

pytestmark = pytest.mark.gpu


def give_up(g, hook, X, W, C, group):
    """One launch whose last block of K's share never gets W; its status and the site where a wait ran out."""
    M, K = X.shape
    assert g.check() == g.GEMM_OK
    st = hook(X.data_ptr(), g.TYPES[X.dtype], W[0].data_ptr(), W[1].data_ptr(), W[2].data_ptr() if W[2] is not None else None,
              C.data_ptr(), M, C.shape[1], K, group, 1 << 20, torch.cuda.current_stream().cuda_stream)
    assert st == g.GEMM_OK
    assert g.check() == g.GEMM_ERR_TIMEOUT
    return g.last_timeout_record() & 0xFF


# K by itself, and over two, four and eight blocks.
@pytest.mark.parametrize("N,K", [(20000, 1024), (9728, 1024), (4096, 2048), (256, 1024), (256, 4096), (130, 16384)])
def test_no_block_of_a_cluster_stores_where_one_gave_up(g, N, K):  # noqa: F811
    W = packed(g, N, K, 64, True, torch.float16, 3)
    X = torch.randn((64, K), device=DEV).half()
    C = torch.full((64, N), 5.0, device=DEV).half()
    assert give_up(g, g.lib().linear_w4_selftest_timeout, X, W, C, 64) == 3
    assert (C == 5.0).all()
    check(g, X, W, N, 64, False)
