"""The 4-bit GEMM's bounded waits, made to run out without a fault.

gemm_mxfp4_selftest_timeout launches the real kernels with loads withheld (all
of them, or the scale tiles' alone while the operands' are under way) and a short
wait budget.  Every role must leave, C stays untouched, gemm_f16_check reports
the timeout, and the next normal call is right.
"""
from __future__ import annotations

import pytest
import torch

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda:0")
# Waits for an empty slot, for scale tiles, for operands and for the accumulator.
SITES = (1, 2, 3, 4)


@pytest.fixture(scope="module")
def g():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    from dense_fp16_gemm_05_gb300 import build as gbuild
    gbuild.build()
    from dense_fp16_gemm_05_gb300 import gemm_f16
    gemm_f16.lib()
    return gemm_f16


# Narrow tiles of 16, 32, 64 and 128 rows, K whole and divided over clusters of 2 to
# 8 CTAs; pair tiles, one per pair and several; K loops shorter than the ring
# (every load is issued before a wait runs out) and longer ones.
@pytest.mark.parametrize("withhold", [1, 2])
@pytest.mark.parametrize("M,N,K", [(1, 256, 512), (1, 4096, 4096), (16, 256, 16384), (30, 512, 2048), (60, 256, 8192),
                                   (300, 4096, 512), (300, 4096, 4096), (1024, 4096, 512), (1024, 4096, 4096),
                                   (2560, 8192, 768)])
def test_waits_run_out_and_context_survives(g, M, N, K, withhold):
    gen = torch.Generator(device=DEV).manual_seed(M + N + K)
    x = torch.randn((M, K), generator=gen, device=DEV, dtype=torch.bfloat16)
    w = torch.randn((N, K), generator=gen, device=DEV, dtype=torch.bfloat16)
    Q, S, V = g.mxfp4_quantize(x, values=True)
    Qw, Sw, Vw = g.mxfp4_quantize(w, values=True)      # values are exact in bf16
    C = torch.full((M, N), 5.0, dtype=torch.float16, device=DEV)
    assert g.check() == g.GEMM_OK
    st = g.lib().gemm_mxfp4_selftest_timeout(Q.data_ptr(), S.data_ptr(), Qw.data_ptr(), Sw.data_ptr(), C.data_ptr(),
                                             M, N, K, withhold, 1 << 20, torch.cuda.current_stream().cuda_stream)
    assert st == g.GEMM_OK
    assert g.check() == g.GEMM_ERR_TIMEOUT
    assert (g.last_timeout_record() & 0xFF) in SITES, hex(g.last_timeout_record())
    assert (C == 5.0).all()
    assert g.check() == g.GEMM_OK
    g.gemm_mxfp4(Q, S, Qw, Sw, C=C, K=K)
    assert g.check() == g.GEMM_OK
    want = V.double() @ Vw.double().t()
    mag = V.double().abs() @ Vw.double().abs().t()
    assert ((C.double() - want).abs() <= 2.0 ** -11 * want.abs() + 2.0 ** -25 + (K / 64 + 16) * 2.0 ** -22 * mag).all()
