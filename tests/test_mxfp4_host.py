"""Refusals and layouts of the MXFP4 entry points that need no GPU."""
from __future__ import annotations

import ctypes

import numpy as np
import pytest
import torch

import mxfp4_reference as ref
from dense_fp16_gemm_05_gb300 import build as gbuild


@pytest.fixture(scope="module")
def g():
    gbuild.build()
    from dense_fp16_gemm_05_gb300 import gemm_f16
    gemm_f16.lib()
    return gemm_f16


def test_entry_points_are_exported_and_declared(g):
    raw = ctypes.CDLL(gbuild.LIB)
    text = open(g.HEADER).read()
    for name in ("mxfp4_quantize", "gemm_mxfp4"):
        assert hasattr(raw, name) and f"int {name}(" in text


@pytest.mark.parametrize("rows,K,type_,trans", [(-1, 32, 0, 0), (4, -32, 0, 0), (2**31, 32, 0, 0), (4, 2**31, 0, 0),
                                                (4, 32, 3, 0), (4, 32, -1, 0), (4, 32, 0, 2)])
def test_quantize_refuses_bad_arguments_before_any_cuda_call(g, rows, K, type_, trans):
    assert g.lib().mxfp4_quantize(None, type_, None, None, None, rows, K, trans, None) == g.GEMM_ERR_INVALID_ARG
    assert g.lib().gemm_f16_last_error_detail()


@pytest.mark.parametrize("M,N,K,relu", [(-1, 8, 32, 0), (8, -8, 32, 0), (8, 8, -1, 0), (2**31, 8, 32, 0),
                                        (8, 2**31, 32, 0), (8, 8, 2**31, 0), (8, 8, 32, 2), (8, 8, 32, -1)])
def test_product_refuses_bad_arguments_before_any_cuda_call(g, M, N, K, relu):
    assert g.lib().gemm_mxfp4(None, None, None, None, None, M, N, K, relu, None) == g.GEMM_ERR_INVALID_ARG


def test_empty_problems_are_no_ops_without_a_gpu(g):
    assert g.lib().mxfp4_quantize(None, 0, None, None, None, 0, 32, 0, None) == g.GEMM_OK
    assert g.lib().mxfp4_quantize(None, 0, None, None, None, 32, 0, 1, None) == g.GEMM_OK
    assert g.lib().gemm_mxfp4(None, None, None, None, None, 0, 8, 32, 0, None) == g.GEMM_OK
    assert g.lib().gemm_mxfp4(None, None, None, None, None, 8, 0, 32, 0, None) == g.GEMM_OK


def test_binding_refuses_wrong_tensors(g):
    x = torch.zeros((4, 64), dtype=torch.float16)
    with pytest.raises(TypeError):
        g.mxfp4_quantize([1.0])
    with pytest.raises(ValueError):
        g.mxfp4_quantize(x.double())
    with pytest.raises(ValueError):
        g.mxfp4_quantize(x[0])
    with pytest.raises(ValueError):
        g.mxfp4_quantize(x.t())
    with pytest.raises(ValueError):
        g.mxfp4_quantize(x, Q=torch.zeros((4, 16), dtype=torch.uint8))
    q, s = (torch.zeros(sh, dtype=torch.uint8) for sh in g.mxfp4_shapes(8, 64))
    with pytest.raises(ValueError):
        g.gemm_mxfp4(q, s, q, s, K=96)
    with pytest.raises(ValueError):
        g.gemm_mxfp4(q, s[:, :, :256], q, s)
    with pytest.raises(ValueError):
        g.gemm_mxfp4(q, s, q, s, C=torch.zeros((8, 8)))
    with pytest.raises(ValueError):
        g.mxfp4_tile_scales(torch.zeros((4, 4)))
    with pytest.raises(ValueError):
        g.mxfp4_row_scales(s, 300, 64)


@pytest.mark.parametrize("rows,K", [(1, 1), (31, 32), (128, 128), (129, 130), (300, 1000)])
def test_scale_tile_order(g, rows, K):
    rng = np.random.default_rng(rows * 1000 + K)
    e = rng.integers(0, 255, (rows, -(-K // 32)), dtype=np.uint8)
    t = g.mxfp4_tile_scales(torch.from_numpy(e))
    assert tuple(t.shape) == g.mxfp4_shapes(rows, K)[1]
    assert np.array_equal(t.numpy(), ref.tile_scales(e))
    assert np.array_equal(g.mxfp4_row_scales(t, rows, K).numpy(), e)


def test_reference_rounding_by_hand():
    x = np.array([[0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 5.1, 7.9, -0.25, -2.6, 4.0] + [0.0] * 20])
    codes, scales = ref.quantize(x)
    assert scales[0, 0] == 127
    want = [0, 1, 1, 2, 2, 4, 4, 6, 6, 0, -3, 4]
    assert ref.decode(codes, scales)[0, :12].tolist() == want
