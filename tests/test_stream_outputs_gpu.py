"""Calls with ``stream=`` while freed memory of the outputs' sizes is still in
use on torch's current stream: the results must not be overwritten by it."""
from __future__ import annotations

import pytest
import torch

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda:0")
H, F, U8 = torch.float16, torch.float32, torch.uint8


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
    gen = torch.Generator(device=DEV).manual_seed(5)

    def half(*shape):
        return torch.randn(shape, generator=gen, device=DEV).half()

    x, w, b = half(64, 512), half(512), half(512)
    A, B, dC = half(64, 512), half(512, 256), half(64, 256)
    qa, qb = g.mxfp4_quantize(A), g.mxfp4_quantize(B, transpose=True)
    _, mean, rstd = g.layer_norm_fwd(x, w, b)
    e4, e4w = (half(r, 512).to(torch.float8_e4m3fn) for r in (64, 256))
    ones = [torch.ones(s, device=DEV) for s in ((64, 4), (2, 4))]
    exps = [torch.full(s, 127, dtype=U8, device=DEV) for s in ((64, 4), (2, 4))]
    Q, K, V = (half(1, 2, 256, 64) for _ in range(3))
    return {
        "mxfp4_quantize": lambda s: g.mxfp4_quantize(x, values=True, stream=s),
        "gemm_mxfp4": lambda s: g.gemm_mxfp4(*qa, *qb, stream=s),
        "layer_norm_fwd": lambda s: g.layer_norm_fwd(x, w, b, stream=s),
        "layer_norm_bwd": lambda s: g.layer_norm_bwd(A, x, mean, rstd, w, stream=s),
        "gemm_f16": lambda s: g.gemm_f16(A, B, stream=s),
        "gemm_f16_t": lambda s: g.gemm_f16_t(dC, B, transb=True, stream=s),
        "relu_backward": lambda s: g.relu_backward(dC, dC.roll(1), stream=s),
        "gemm_fp8_block_scaled": lambda s: g.gemm_fp8_block_scaled(e4, ones[0], e4w, ones[1], stream=s),
        "gemm_mxfp8_block_scaled": lambda s: g.gemm_mxfp8_block_scaled(e4, exps[0], e4w, exps[1], stream=s),
        "attention_fwd": lambda s: g.attention_fwd(Q, K, V, stream=s),
    }


@pytest.mark.parametrize("name", ["mxfp4_quantize", "gemm_mxfp4", "layer_norm_fwd", "layer_norm_bwd", "gemm_f16",
                                  "gemm_f16_t", "relu_backward", "gemm_fp8_block_scaled", "gemm_mxfp8_block_scaled",
                                  "attention_fwd"])
def test_pending_work_on_the_current_stream_does_not_reach_the_outputs(g, name):
    call = calls(g)[name]
    want = call(None)
    want = want if isinstance(want, tuple) else (want,)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    torch.cuda.empty_cache()
    # blocks of the outputs' sizes, freed with a fill still queued behind some 10 ms
    blocks = [torch.empty_like(t) for t in want]
    torch.cuda._sleep(20_000_000)
    for t in blocks:
        t.view(U8).fill_(0x55)
    del blocks, t
    got = call(side)
    got = got if isinstance(got, tuple) else (got,)
    torch.cuda.synchronize()
    assert g.check() == g.GEMM_OK
    for a, b in zip(got, want):
        # scale bytes of rows that a tile does not have are not written
        if name == "mxfp4_quantize" and a.dim() == 3:
            a, b = g.mxfp4_row_scales(a, 64, 512), g.mxfp4_row_scales(b, 64, 512)
        assert torch.equal(a, b)


def test_host_tensors_are_refused_on_a_given_stream(g):
    side = torch.cuda.Stream()
    a = torch.zeros((8, 8), dtype=H)
    with pytest.raises(Exception):
        g.gemm_f16(a, a, stream=side)
    assert g.check() == g.GEMM_OK


def test_inputs_dropped_right_after_the_call(g):
    # the next allocations on the current stream would land in their memory
    gen = torch.Generator(device=DEV).manual_seed(6)
    base = [torch.randn((64, 512), generator=gen, device=DEV).half() for _ in range(2)]
    _, mean, rstd = g.layer_norm_fwd(base[1])
    want = (*g.mxfp4_quantize(base[0], values=True)[::2], g.layer_norm_fwd(base[0])[0],
            *g.layer_norm_bwd(*base, mean, rstd))
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    with torch.cuda.stream(side):
        torch.cuda._sleep(20_000_000)

    def fresh(t):
        return torch.empty_like(t).copy_(t)

    got = []
    inputs = [[fresh(base[0])], [fresh(base[0])], [fresh(t) for t in (*base, mean, rstd)]]
    torch.cuda.current_stream().synchronize()
    got += g.mxfp4_quantize(*inputs.pop(0), values=True, stream=side)[::2]
    got.append(g.layer_norm_fwd(*inputs.pop(0), stream=side)[0])
    got += g.layer_norm_bwd(*inputs.pop(0), stream=side)
    for _ in range(6):
        for t in (base[0], mean):
            torch.full_like(t, 7.0)
    torch.cuda.synchronize()
    assert g.check() == g.GEMM_OK and all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("name", ["mxfp4_quantize", "layer_norm_bwd", "gemm_f16", "attention_fwd"])
@pytest.mark.parametrize("kind", ["null", "raw"])
def test_raw_handles(g, name, kind):
    call = calls(g)[name]
    want = call(None)
    want = want if isinstance(want, tuple) else (want,)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    got = call(0 if kind == "null" else side.cuda_stream)
    got = got if isinstance(got, tuple) else (got,)
    if name == "layer_norm_bwd":
        assert g._launch_stream(0, DEV) == torch.cuda.default_stream(DEV)
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        if name == "mxfp4_quantize" and a.dim() == 3:
            a, b = g.mxfp4_row_scales(a, 64, 512), g.mxfp4_row_scales(b, 64, 512)
        assert torch.equal(a, b)
