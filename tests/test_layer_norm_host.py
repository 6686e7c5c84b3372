"""Refusals of the layer norm entry points that need no GPU."""
from __future__ import annotations

import ctypes

import pytest
import torch

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
    for name in ("layer_norm_fwd", "layer_norm_bwd", "layer_norm_bwd_workspace"):
        assert hasattr(raw, name) and f"{name}(" in text


@pytest.mark.parametrize("rows,dim,eps,xt,wt", [(-1, 8, 0.0, 0, 0), (8, -1, 0.0, 0, 0), (2**31, 8, 0.0, 0, 0),
                                                (8, 2**31, 0.0, 0, 0), (8, 8, -1.0, 0, 0), (8, 8, float("nan"), 0, 0),
                                                (8, 8, float("inf"), 0, 0), (8, 8, 0.0, 3, 2), (8, 8, 0.0, 0, 1),
                                                (8, 8, 0.0, 2, 0), (8, 8, 0.0, 0, -1)])
def test_forward_refuses_bad_arguments_before_any_cuda_call(g, rows, dim, eps, xt, wt):
    st = g.lib().layer_norm_fwd(None, None, None, None, None, None, rows, dim, eps, xt, wt, None)
    assert st == g.GEMM_ERR_INVALID_ARG


def test_null_buffers_are_refused_before_any_cuda_call(g):
    L = g.lib()
    assert L.layer_norm_fwd(None, None, None, 16, None, None, 2, 8, 0.0, 0, 0, None) == g.GEMM_ERR_INVALID_ARG
    assert L.layer_norm_bwd(None, 16, None, 16, 16, 16, None, None, 2, 8, 0, 0, None, 0, None) == g.GEMM_ERR_INVALID_ARG
    # dgamma without dbeta
    assert L.layer_norm_bwd(16, 16, None, 16, 16, 16, 16, None, 2, 8, 0, 0, 16, 0, None) == g.GEMM_ERR_INVALID_ARG


def test_empty_problems_are_no_ops_without_a_gpu(g):
    L = g.lib()
    assert L.layer_norm_fwd(None, None, None, None, None, None, 0, 8, 0.0, 0, 0, None) == g.GEMM_OK
    assert L.layer_norm_fwd(None, None, None, None, None, None, 8, 0, 0.0, 0, 0, None) == g.GEMM_OK
    assert L.layer_norm_bwd(*[None] * 8, 8, 0, 0, 0, None, 0, None) == g.GEMM_OK
    assert L.layer_norm_bwd(*[None] * 8, 0, 8, 0, 0, None, 0, None) == g.GEMM_OK


def test_binding_refuses_wrong_tensors(g):
    x = torch.zeros((4, 16), dtype=torch.float16)
    w = torch.ones(16, dtype=torch.float16)
    r = torch.zeros(4)
    with pytest.raises(TypeError):
        g.layer_norm_fwd([1.0])
    for bad in (x.double(), x.t(), x[:, :8]):
        with pytest.raises(ValueError):
            g.layer_norm_fwd(bad)
    for gamma, beta in ((w[:8], None), (w.bfloat16(), None), (w, w.float()), (None, w.double())):
        with pytest.raises(ValueError):
            g.layer_norm_fwd(x, gamma, beta)
    with pytest.raises(ValueError):
        g.layer_norm_fwd(x, w, w, Y=x.float())
    with pytest.raises(ValueError):
        g.layer_norm_bwd(x.float(), x, r, r)
    with pytest.raises(ValueError):
        g.layer_norm_bwd(x, x, r.half(), r)
    with pytest.raises(ValueError):
        g.layer_norm_bwd(x, x, r, r, wtype=torch.bfloat16)
