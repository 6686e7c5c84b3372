"""Without the module of csrc/binding.cpp the calls that it shortens go through ctypes: on
the CPU, up to the library's own refusal of host memory."""
from __future__ import annotations

import pytest
import torch

from dense_fp16_gemm_05_gb300 import build as gbuild


@pytest.fixture
def g(monkeypatch, tmp_path):
    gbuild.build()
    from dense_fp16_gemm_05_gb300 import gemm_f16
    gemm_f16.lib()
    monkeypatch.setattr(gemm_f16, "_binding", None)
    return gemm_f16


@pytest.mark.parametrize("there", [False, True])
def test_calls_without_the_module(g, monkeypatch, tmp_path, there):
    path = tmp_path / "_binding.so"
    if there:
        path.write_bytes(b"not a module of this Python")
    monkeypatch.setattr(g._build, "binding_path", lambda: str(path))
    x = torch.zeros((4, 128), dtype=torch.float16)
    with pytest.warns(RuntimeWarning, match="ctypes"):
        with pytest.raises(ValueError):
            g.rms_norm_fwd(x, gamma=x)
    # once; what follows goes the long way without a word, and refuses as it does
    with pytest.raises(ValueError):
        g.rms_norm_fp8(x, residual=x[:2])
    with pytest.raises(ValueError):
        g.rms_norm_bwd(x, x, torch.zeros(3))
    with pytest.raises(ValueError):
        g.fp8_quantize(x, block_rows=5)
    with pytest.raises(ValueError):
        g.dropout(x, 1.0, 0)
    with pytest.raises(ValueError):
        g.linear_w4(x, torch.zeros(1, dtype=torch.uint8), x)


def test_every_shortened_call_has_a_stand_in(g):
    module = g._short()
    if module is g._LongWay:
        pytest.skip("the module is not built here")
    for name in ("rms_norm_fwd", "rms_norm_fp8", "rms_norm_bwd", "fp8_quantize", "dropout", "linear_w4"):
        assert callable(getattr(module, name)) and getattr(g._LongWay, name)(1, 2, 3) is None


def test_the_library_itself_is_still_asked_for(g, monkeypatch, tmp_path):
    monkeypatch.setattr(g, "_lib", None)
    monkeypatch.setattr(g._build, "LIB", str(tmp_path / "none.so"))
    with pytest.raises(g.LibraryNotBuilt):
        g.rms_norm_fwd(torch.zeros((4, 128), dtype=torch.float16))
