"""The binding's short way to a new tensor, on the CPU with stand-ins: torch.empty
serves where torch's function is missing or has changed."""
from __future__ import annotations

import types

import pytest
import torch

from dense_fp16_gemm_05_gb300 import gemm_f16 as g

DEVICE = types.SimpleNamespace(index=0)


def gone(*args):
    raise AttributeError("no such name")


def other_arguments(size, stride, dtype, device):
    raise AssertionError("not reached")


def other_meaning(size, stride, dtype):
    return torch.empty(6, dtype=dtype)


@pytest.fixture
def plain(monkeypatch):
    monkeypatch.setattr(g, "_current_device", lambda: 0)
    empty = torch.empty
    monkeypatch.setattr(torch, "empty", lambda shape, dtype, device=None: empty(tuple(shape), dtype=dtype))
    monkeypatch.setattr(g, "_empty_strided_cuda", False)


@pytest.mark.parametrize("function", [gone, other_arguments, other_meaning])
def test_a_changed_function_is_not_used(plain, monkeypatch, function):
    monkeypatch.setattr(torch._C._dynamo.guards, "_empty_strided_cuda", function)
    for shape in ((4, 5), (7,), (2, 3, 4), ()):
        t = g._new(shape, torch.float32, DEVICE)
        assert tuple(t.shape) == shape and t.dtype == torch.float32 and t.is_contiguous()
    assert g._empty_strided_cuda is None


def test_the_function_is_used_where_it_does_what_is_needed(plain, monkeypatch):
    class Made:
        def __init__(self, size, stride, dtype):
            self.shape, self._stride, self.dtype, self.device = size, stride, dtype, torch.device("cuda", 0)

        def stride(self):
            return self._stride

    monkeypatch.setattr(torch._C._dynamo.guards, "_empty_strided_cuda", Made)
    t = g._new((4, 5), torch.float32, DEVICE)
    assert isinstance(t, Made) and t.shape == (4, 5) and t.stride() == (5, 1)
    assert g._new((2, 3, 4), torch.uint8, DEVICE).stride() == (12, 4, 1)
