"""GPU tests of the order of the sums in products with 4-bit weights: it goes by the
sizes and the GPU alone, so equal values give equal bits wherever X lies."""
from __future__ import annotations

import pytest
import torch

from test_linear_w4_gpu import DEV, DTYPES, check, g, packed  # noqa: F401  (g: a fixture)

pytestmark = pytest.mark.gpu


# Sizes of every kernel; a division of the work that counts what it takes to copy X
# differs in most of them between X on the 16-byte grid and off it.
@pytest.mark.parametrize("xt", ["fp16", "bf16"])
@pytest.mark.parametrize("M,N,K,group", [
    (1, 4096, 4096, 32), (4, 4096, 8192, 128), (8, 4096, 11008, 64), (9, 3914, 3032, 128), (12, 4096, 4096, 32),
    (15, 488, 1056, 128), (17, 2048, 4096, 64), (28, 1273, 1712, 64), (24, 4096, 4096, 128), (20, 16384, 4096, 64),
    (26, 3873, 5616, 64), (32, 16384, 8192, 32), (64, 1024, 8192, 128), (3, 4096, 4001, 64), (30, 4099, 4097, 32)])
def test_the_place_of_x_does_not_change_a_bit(g, M, N, K, group, xt):  # noqa: F811
    W = packed(g, N, K, group, group != 64, DTYPES[xt], M + N + K)
    gen = torch.Generator().manual_seed(N)
    X = torch.randn((M, K), generator=gen).to(DTYPES[xt]).to(DEV)
    want = check(g, X, W, N, group, relu=False)
    for by in (1, 2, 8, 13):
        flat = torch.full((M * K + 32,), float("nan"), dtype=X.dtype, device=DEV)
        there = flat[by:by + M * K].reshape(M, K)
        there.copy_(X)
        assert torch.equal(g.linear_w4(there, *W, N=N, group=group), want), by
    assert g.check() == g.GEMM_OK


# Seven units of 128 columns to a block, alone and in clusters: seven ways of a strip.
@pytest.mark.parametrize("M,N,K", [(1, 300, 896), (8, 4096, 896), (16, 512, 880), (30, 1024, 850), (8, 2048, 1792),
                                   (16, 1000, 3584), (5, 1024, 7168), (16, 200, 7050)])
def test_seven_units_of_a_block(g, M, N, K):  # noqa: F811
    W = packed(g, N, K, 64, True, torch.bfloat16, M + N + K)
    X = torch.randn((M, K), device=DEV).bfloat16()
    check(g, X, W, N, 64, relu=M % 2 == 0)
