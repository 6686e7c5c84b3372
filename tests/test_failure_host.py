"""Refusals of the timeout test hooks before any CUDA call."""
from __future__ import annotations

import ctypes

import pytest

from dense_fp16_gemm_05_gb300 import build as gbuild


@pytest.fixture(scope="module")
def g():
    gbuild.build()
    from dense_fp16_gemm_05_gb300 import gemm_f16
    gemm_f16.lib()
    return gemm_f16


def test_hooks_are_exported_and_declared(g):
    raw = ctypes.CDLL(gbuild.LIB)
    text = open(g.HEADER).read()
    for name in ("gemm_mxfp4_selftest_timeout", "layer_norm_bwd_selftest_timeout"):
        assert hasattr(raw, name) and f"int {name}(" in text


@pytest.mark.parametrize("M,N,K,withhold,cycles", [(0, 8, 32, 1, 1 << 20), (8, 8, 0, 1, 1 << 20), (8, 8, 32, 0, 1 << 20),
                                                   (8, 8, 32, 3, 1 << 20), (8, 8, 32, 1, 100), (8, 8, 32, 2, 1 << 40)])
def test_product_hook_refuses(g, M, N, K, withhold, cycles):
    st = g.lib().gemm_mxfp4_selftest_timeout(None, None, None, None, None, M, N, K, withhold, cycles, None)
    assert st == g.GEMM_ERR_INVALID_ARG


@pytest.mark.parametrize("rows,dim,cycles", [(0, 1024, 1 << 20), (8, 0, 1 << 20), (8, 1024, 100), (8, 1024, 1 << 40),
                                             (-1, 1024, 1 << 20)])
def test_norm_hook_refuses(g, rows, dim, cycles):
    st = g.lib().layer_norm_bwd_selftest_timeout(None, None, None, None, None, rows, dim, 0, cycles, None)
    assert st == g.GEMM_ERR_INVALID_ARG
