"""4-bit linear on types and sizes outside its gradients' GEMMs: what needs no
gradient, or only the one that the other operand allows, is answered."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import mxfp4_reference as ref

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda:0")
H, BF, F = torch.float16, torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def ag():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    from dense_fp16_gemm_05_gb300 import build as gbuild
    gbuild.build()
    from dense_fp16_gemm_05_gb300 import autograd
    return autograd


def operands(M, N, K, ta, tb):
    gen = torch.Generator().manual_seed(M + N + K)
    A, B = torch.randn((M, K), generator=gen).to(ta), torch.randn((K, N), generator=gen).to(tb)
    a = ref.decode(*ref.quantize(A.double().numpy()))[:, :K]
    b = ref.decode(*ref.quantize(B.t().double().numpy()))[:, :K]
    return A.to(DEV), B.to(DEV), a, b


def check_output(C, a, b, K):
    want, mag = ref.product(a, b, False)
    assert np.all(np.abs(C.detach().cpu().double().numpy() - want) <= ref.product_tolerance(want, mag, K))


@pytest.mark.parametrize("K,ta,tb", [(36, H, H), (50, BF, BF), (64, F, F), (1, BF, F)])
def test_without_gradients(ag, K, ta, tb):
    A, B, a, b = operands(20, 16, K, ta, tb)
    check_output(ag.linear_mxfp4(A, B), a, b, K)
    A.requires_grad_()
    with torch.no_grad():
        check_output(ag.linear_mxfp4(A, B), a, b, K)


@pytest.mark.parametrize("which", ["A", "B"])
def test_the_gradient_that_the_other_operand_allows(ag, which):
    A, B, a, b = operands(24, 16, 64, F if which == "A" else H, BF if which == "B" else H)
    (A if which == "A" else B).requires_grad_()
    C = ag.linear_mxfp4(A, B)
    check_output(C, a, b, 64)
    dC = torch.randn((24, 16), generator=torch.Generator().manual_seed(1)).half()
    C.backward(dC.to(DEV))
    got, x, y = (A.grad, dC.double().numpy(), b) if which == "A" else (B.grad, a.T, dC.double().numpy())
    want = x @ y
    # a rounding to fp16 and one to the operand's type; fp32 sums of up to 24 exact products
    rel = 2.0 ** -11 + (2.0 ** -8 if got.dtype == BF else 2.0 ** -24)
    tol = rel * np.abs(want) + 2.0 ** -25 + 34 * 2.0 ** -24 * (np.abs(x) @ np.abs(y))
    assert got.dtype == (F if which == "A" else BF)
    assert np.all(np.abs(got.cpu().double().numpy() - want) <= 1.01 * tol)
