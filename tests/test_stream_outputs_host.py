"""Where a call with ``stream=`` allocates what it hands back, on the CPU: every
output must come from the pool of the stream that writes it.  The streams, the
launches and the allocator are stand-ins."""
from __future__ import annotations

import contextlib
import ctypes
import types

import pytest
import torch

from dense_fp16_gemm_05_gb300 import gemm_f16 as g

LAUNCH, CURRENT = object(), object()
H, F, U8 = torch.float16, torch.float32, torch.uint8


@pytest.fixture
def made(monkeypatch):
    """Allocations as (tensor, stream they were made under), and recorded uses."""
    log = types.SimpleNamespace(allocated=[], recorded=[])
    under = [CURRENT]

    @contextlib.contextmanager
    def stream(s):
        under.append(s)
        yield
        under.pop()

    empty = torch.empty

    def new(*args, **kw):
        t = empty(*args, **kw)
        log.allocated.append((t, under[-1]))
        return t

    class Lib:
        def __getattr__(self, name):
            return lambda *args: g.GEMM_OK

    monkeypatch.setattr(torch.cuda, "stream", stream)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: CURRENT)
    monkeypatch.setattr(torch, "empty", new)
    monkeypatch.setattr(torch, "empty_like", lambda t: new(t.shape, dtype=t.dtype))
    monkeypatch.setattr(torch.Tensor, "record_stream", lambda t, s: log.recorded.append((t, s)))
    monkeypatch.setattr(g, "_on_gpu", lambda device: True)
    monkeypatch.setattr(g, "_launch_stream", lambda stream, device: LAUNCH)
    monkeypatch.setattr(g, "_stream_handle", lambda stream, device: 0)
    monkeypatch.setattr(g, "_device_scope", lambda device: contextlib.nullcontext())
    monkeypatch.setattr(g, "_lib", Lib())
    return log


def zeros(shape, dtype):
    return torch.zeros(shape, dtype=dtype)


def codes(rows, K):
    return [zeros(s, U8) for s in g.mxfp4_shapes(rows, K)]


CALLS = {
    "mxfp4_quantize": lambda s: g.mxfp4_quantize(zeros((4, 64), H), values=True, stream=s),
    "gemm_mxfp4": lambda s: g.gemm_mxfp4(*codes(4, 64), *codes(8, 64), stream=s),
    "layer_norm_fwd": lambda s: g.layer_norm_fwd(zeros((4, 64), H), zeros(64, H), zeros(64, H), stream=s),
    "layer_norm_bwd": lambda s: g.layer_norm_bwd(zeros((4, 64), H), zeros((4, 64), H), zeros(4, F), zeros(4, F),
                                                 zeros(64, H), workspace=zeros(16, F), stream=s),
    "gemm_f16": lambda s: g.gemm_f16(zeros((4, 8), H), zeros((8, 8), H), stream=s),
    "gemm_f16_t": lambda s: g.gemm_f16_t(zeros((4, 8), H), zeros((8, 8), H), transb=True, stream=s),
    "relu_backward": lambda s: g.relu_backward(zeros((4, 8), H), zeros((4, 8), H), stream=s),
    "gemm_fp8_block_scaled": lambda s: g.gemm_fp8_block_scaled(zeros((4, 128), U8), zeros((4, 1), F),
                                                               zeros((8, 128), U8), zeros((1, 1), F), stream=s),
    "gemm_mxfp8_block_scaled": lambda s: g.gemm_mxfp8_block_scaled(zeros((4, 128), U8), zeros((4, 1), U8),
                                                                   zeros((8, 128), U8), zeros((1, 1), U8), stream=s),
    "attention_fwd": lambda s: g.attention_fwd(*[zeros((1, 1, 4, 64), H)] * 3, stream=s),
    "tma_box_image": lambda s: g.tma_box_image(zeros((4, 64), H), 4, 0, 0, stream=s),
}


@pytest.mark.parametrize("name", list(CALLS))
def test_outputs_come_from_the_launch_streams_pool(made, name):
    out = CALLS[name](LAUNCH)
    outputs = [t for t in (out if isinstance(out, tuple) else (out,)) if t is not None]
    assert outputs
    for t in outputs:
        assert [s for u, s in made.allocated if u is t] == [LAUNCH]
        # and are handed out on the current stream
        assert any(u is t and s is CURRENT for u, s in made.recorded)


@pytest.mark.parametrize("name", list(CALLS))
def test_without_a_stream_nothing_is_recorded(made, name):
    CALLS[name](None)
    assert made.allocated and all(s is CURRENT for _, s in made.allocated) and not made.recorded


def _inputs(monkeypatch):
    """Every tensor that zeros() makes for a call."""
    kept = []
    plain = zeros

    def keep(shape, dtype):
        t = plain(shape, dtype)
        kept.append(t)
        return t

    monkeypatch.setitem(globals(), "zeros", keep)
    return kept


@pytest.mark.parametrize("name", ["mxfp4_quantize", "gemm_mxfp4", "layer_norm_fwd", "layer_norm_bwd"])
def test_inputs_are_recorded_on_the_launch_stream(made, monkeypatch, name):
    # a temporary passed to the call is dropped before the launch stream has read it
    kept = _inputs(monkeypatch)
    CALLS[name](LAUNCH)
    assert kept
    for t in kept:
        assert any(u is t and s is LAUNCH for u, s in made.recorded)


def test_a_null_handle_is_the_default_stream(monkeypatch):
    monkeypatch.setattr(torch.cuda, "default_stream", lambda device=None: LAUNCH)
    monkeypatch.setattr(torch.cuda, "ExternalStream", lambda handle, device=None: (handle, device))
    assert g._launch_stream(0, "cuda:0") is LAUNCH
    assert g._launch_stream(ctypes.c_void_p(8).value, "cuda:0") == (8, "cuda:0")
