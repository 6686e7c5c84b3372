"""GPU tests that the calls give the same without the module of csrc/binding.cpp as with it."""
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


def calls(g):
    gen = torch.Generator().manual_seed(3)
    x, r, dy = (torch.randn((7, 5, 264), generator=gen).bfloat16().to(DEV) for _ in range(3))
    w = (1 + 0.2 * torch.randn(264, generator=gen)).to(DEV)
    flat = x.reshape(35, 264)
    offset = torch.tensor([11], device=DEV)
    W = g.w4_quantize(torch.randn((48, 264), generator=gen).to(DEV), 64, True, stype=torch.bfloat16)
    Y, H, rstd = g.rms_norm_fwd(x, w, residual=r)
    out = [Y, H, rstd, *g.rms_norm_fwd(x, None, eps=1e-5, stats=False)[:2]]
    for pow2 in (False, True):
        out += [*g.rms_norm_fp8(x, w, residual=r, pow2=pow2), *g.rms_norm_fp8(x, pow2=pow2),
                *g.fp8_quantize(flat, 1, pow2), *g.fp8_quantize(flat, 128, pow2)]
    out += [*g.rms_norm_bwd(dy, H, rstd, w, dH=r), g.rms_norm_bwd(dy, H, rstd, weights=False)[0]]
    out += [g.dropout(x, 0.25, 5, 7, residual=r), g.dropout(x, 0.25, 5, offset)]
    out += [g.linear_w4(flat[:9], *W, N=48, group=64, relu=True), g.linear_w4(flat, *W, group=64)]
    assert g.check() == g.GEMM_OK
    return out


def test_the_same_without_the_module(g, monkeypatch, tmp_path):
    want = calls(g)
    assert g._binding is not None and g._binding is not g._LongWay
    monkeypatch.setattr(g, "_binding", None)
    monkeypatch.setattr(g._build, "binding_path", lambda: str(tmp_path / "_binding.so"))
    with pytest.warns(RuntimeWarning, match="ctypes"):
        got = calls(g)
    assert g._binding is g._LongWay
    assert len(got) == len(want)
    for a, b in zip(got, want):
        assert a.dtype == b.dtype and a.shape == b.shape
        assert torch.equal(a.contiguous().view(torch.uint8), b.contiguous().view(torch.uint8))
