"""Offsets past 2^31 elements in the MXFP4 and layer norm kernels, against the
same rows computed in small calls."""
from __future__ import annotations

import pytest
import torch

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


@pytest.fixture(autouse=True)
def release():
    yield
    torch.cuda.empty_cache()


def big_rows(rows, dim, dtype):
    """Rows that differ, without a generator's time: a few random rows, shifted and scaled."""
    gen = torch.Generator(device=DEV).manual_seed(1)
    base = torch.randn((64, dim), generator=gen, device=DEV, dtype=torch.float32)
    x = torch.empty((rows, dim), dtype=dtype, device=DEV)
    for r in range(0, rows, 64):
        n = min(64, rows - r)
        x[r:r + n] = (base[:n] * (1 + (r % 4096) / 4096)).to(dtype)
    return x


ROWS, DIM = 66000, 32776      # 2.16e9 elements, past 2^31; 16-byte rows, no power of 2
SPOTS = [(0, 128), (32768, 32896), (65408, 65536), (65920, 66000)]


def test_quantize_rows_past_2_31_elements(g):
    x = big_rows(ROWS, DIM, torch.float16)
    Q, S, V = g.mxfp4_quantize(x, values=True)
    assert g.check() == g.GEMM_OK
    for a, b in SPOTS:
        q, s, v = g.mxfp4_quantize(x[a:b].contiguous(), values=True)
        assert torch.equal(Q[a:b], q) and torch.equal(V[a:b], v)
        assert torch.equal(g.mxfp4_row_scales(S[a // 128:-(-b // 128)].contiguous(), b - a, DIM),
                           g.mxfp4_row_scales(s, b - a, DIM))


def test_quantize_columns_past_2_31_elements(g):
    x = big_rows(DIM, ROWS, torch.float16)      # (K, rows)
    Q, S = g.mxfp4_quantize(x, transpose=True)
    assert g.check() == g.GEMM_OK
    for a, b in SPOTS:
        q, s = g.mxfp4_quantize(x[:, a:b].contiguous(), transpose=True)
        assert torch.equal(Q[a:b], q)
        assert torch.equal(g.mxfp4_row_scales(S[a // 128:-(-b // 128)].contiguous(), b - a, DIM),
                           g.mxfp4_row_scales(s, b - a, DIM))


def test_product_with_output_past_2_31_elements(g):
    K = 96
    x = big_rows(ROWS, K, torch.bfloat16)
    w = big_rows(DIM, K, torch.bfloat16)
    Q, S, V = g.mxfp4_quantize(x, values=True)
    Qw, Sw, Vw = g.mxfp4_quantize(w, values=True)
    C = g.gemm_mxfp4(Q, S, Qw, Sw)
    assert g.check() == g.GEMM_OK
    for a, b in SPOTS:
        # the same tiles' sums in a smaller call (rows a .. b of 128 fill tiles alike)
        want = V[a:b].double() @ Vw.double().t()
        mag = V[a:b].double().abs() @ Vw.double().abs().t()
        tol = 2.0 ** -11 * want.abs() + 2.0 ** -25 + (K / 64 + 16) * 2.0 ** -22 * mag
        assert ((C[a:b].double() - want).abs() <= tol).all()


@pytest.mark.parametrize("dim", [32776, 16384])
def test_layer_norm_past_2_31_elements(g, dim):
    rows = ROWS * 32776 // dim
    x = big_rows(rows, dim, torch.float16)
    w = torch.linspace(0.5, 1.5, dim, device=DEV).half()
    b = torch.linspace(-1, 1, dim, device=DEV).half()
    Y, mean, rstd = g.layer_norm_fwd(x, w, b)
    spots = [(0, 64), (rows // 2, rows // 2 + 64), (rows - 64, rows)]
    for s, e in spots:
        y, m, r = g.layer_norm_fwd(x[s:e].contiguous(), w, b)
        assert torch.equal(Y[s:e], y) and torch.equal(mean[s:e], m) and torch.equal(rstd[s:e], r)
    dX, dg, db = g.layer_norm_bwd(Y, x, mean, rstd, w)
    assert g.check() == g.GEMM_OK
    for s, e in spots:
        dx, _, _ = g.layer_norm_bwd(Y[s:e].contiguous(), x[s:e].contiguous(), mean[s:e].contiguous(),
                                    rstd[s:e].contiguous(), w)
        assert torch.equal(dX[s:e], dx)
    # the column sums over all rows, in pieces, in 64 bits
    want = torch.zeros(dim, dtype=torch.float64, device=DEV)
    mag = torch.zeros_like(want)
    for r in range(0, rows, 4096):
        y = Y[r:r + 4096].double()
        want += y.sum(0)
        mag += y.abs().sum(0)
    # at most rows / 128 terms one by one and 608 parts, each sum off by half a step
    tol = (rows / 128 + 64) * 2.0 ** -24 * mag + 2.0 ** -11 * want.abs() + 2.0 ** -24
    # Sums past binary16's largest number (65504, and half a step) are infinities.
    over = want.abs() - tol > 65520
    sure = (want.abs() + tol < 65520) | over
    assert torch.equal(torch.isinf(db) & sure, over) and (torch.sign(db) == torch.sign(want))[over].all()
    inside = sure & ~over
    assert inside.any() and ((db.double() - want).abs() <= tol)[inside].all()
