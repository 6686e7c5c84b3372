"""Refusals of the feed-forward layer's functions that need no GPU."""
from __future__ import annotations

import pytest
import torch

from dense_fp16_gemm_05_gb300 import build as gbuild


@pytest.fixture(scope="module")
def ag():
    gbuild.build()
    from dense_fp16_gemm_05_gb300 import autograd, gemm_f16
    gemm_f16.lib()
    return autograd


@pytest.mark.parametrize("a,b", [((4, 40), (48, 8)), ((4, 33), (64, 8)), ((4, 64), (63, 8)), ((4, 64), (96, 8))])
def test_four_bit_linear_refuses_inner_sizes_that_differ(ag, a, b):
    # also those that fill the same number of blocks of 32
    with pytest.raises(ValueError, match="inner sizes differ"):
        ag.linear_mxfp4(torch.zeros(a, dtype=torch.float16), torch.zeros(b, dtype=torch.float16))
