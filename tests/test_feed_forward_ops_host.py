"""Refusals of the operators around a feed-forward block, and their layouts, that need no GPU."""
from __future__ import annotations

import ctypes

import pytest
import torch

import feed_forward_reference as ref
from dense_fp16_gemm_05_gb300 import build as gbuild

H, F, U8 = torch.float16, torch.float32, torch.uint8


@pytest.fixture(scope="module")
def g():
    gbuild.build()
    from dense_fp16_gemm_05_gb300 import gemm_f16
    gemm_f16.lib()
    return gemm_f16


def test_entry_points_are_exported_and_declared(g):
    raw = ctypes.CDLL(gbuild.LIB)
    text = open(g.HEADER).read()
    for name in ("rms_norm_fwd", "rms_norm_fp8", "rms_norm_bwd", "rms_norm_bwd_workspace", "fp8_quantize",
                 "dropout_philox", "w4_quantize", "linear_w4"):
        assert hasattr(raw, name) and f"{name}(" in text


@pytest.mark.parametrize("counter,key,want", [
    ([0] * 4, [0] * 2, [0x6627E8D5, 0xE169C58D, 0xBC57AC4C, 0x9B00DBD8]),
    ([0xFFFFFFFF] * 4, [0xFFFFFFFF] * 2, [0x408F276D, 0x41C83B0E, 0xA20BC7C6, 0x6D5451FD]),
    ([0x243F6A88, 0x85A308D3, 0x13198A2E, 0x03707344], [0xA4093822, 0x299F31D0],
     [0xD16CFE09, 0x94FDCCEB, 0x5001E420, 0x24126EA1])])
def test_reference_generator_gives_the_published_words(counter, key, want):
    # known answers of Philox4x32-10 (the paper's Random123 distribution)
    assert ref.philox_words(counter, key) == want


BAD_NORM = [(-1, 8, 0.0, 0, 0), (8, -1, 0.0, 0, 0), (2**31, 8, 0.0, 0, 0), (8, 2**31, 0.0, 0, 0), (8, 8, -1.0, 0, 0),
            (8, 8, float("nan"), 0, 0), (8, 8, float("inf"), 0, 0), (8, 8, 0.0, 3, 2), (8, 8, 0.0, 0, 1),
            (8, 8, 0.0, 2, 0), (8, 8, 0.0, 0, -1)]


@pytest.mark.parametrize("rows,dim,eps,xt,wt", BAD_NORM)
def test_rms_norm_refuses_bad_arguments_before_any_cuda_call(g, rows, dim, eps, xt, wt):
    L = g.lib()
    assert L.rms_norm_fwd(16, None, None, None, 16, None, rows, dim, eps, xt, wt, None) == g.GEMM_ERR_INVALID_ARG
    assert L.rms_norm_fp8(16, None, None, None, 16, 16, None, rows, dim, eps, xt, wt, 0, None) == g.GEMM_ERR_INVALID_ARG


def test_rms_norm_null_buffers(g):
    L, bad = g.lib(), g.GEMM_ERR_INVALID_ARG
    assert L.rms_norm_fwd(None, None, None, None, 16, None, 2, 8, 0.0, 0, 0, None) == bad
    assert L.rms_norm_fwd(16, None, None, None, None, None, 2, 8, 0.0, 0, 0, None) == bad
    # a residual without a place for the stream, and the other way round
    assert L.rms_norm_fwd(16, 16, None, None, 32, None, 2, 8, 0.0, 0, 0, None) == bad
    assert L.rms_norm_fwd(16, None, None, 16, 32, None, 2, 8, 0.0, 0, 0, None) == bad
    assert L.rms_norm_fp8(16, None, None, None, None, 16, None, 2, 8, 0.0, 0, 0, 0, None) == bad
    assert L.rms_norm_fp8(16, None, None, None, 16, None, None, 2, 8, 0.0, 0, 0, 0, None) == bad
    assert L.rms_norm_fp8(16, None, None, None, 16, 16, None, 2, 8, 0.0, 0, 0, 2, None) == bad
    assert L.rms_norm_bwd(None, 16, None, 16, None, 16, None, 2, 8, 0, 0, None, 0, None) == bad
    assert L.rms_norm_bwd(16, 16, None, None, None, 16, None, 2, 8, 0, 0, None, 0, None) == bad


def test_other_entry_points_refuse_bad_arguments_before_any_cuda_call(g):
    L, bad = g.lib(), g.GEMM_ERR_INVALID_ARG
    for rows, K, block, pow2, t in ((-1, 8, 1, 0, 0), (8, 2**31, 1, 0, 0), (8, 8, 64, 0, 0), (8, 8, 1, 2, 0),
                                    (8, 8, 1, 0, 3), (2**31 - 1, 256, 1, 0, 0)):
        assert L.fp8_quantize(16, t, 16, 16, rows, K, block, pow2, None) == bad
    assert L.fp8_quantize(None, 0, 16, 16, 8, 8, 1, 0, None) == bad
    for n, t, p in ((-1, 0, 0.5), (8, 3, 0.5), (8, 0, 1.0), (8, 0, -0.5), (8, 0, float("nan")), (2**62, 0, 0.5)):
        assert L.dropout_philox(16, None, 16, n, t, p, 0, 0, None, None) == bad
    assert L.dropout_philox(None, None, 16, 8, 0, 0.5, 0, 0, None, None) == bad
    for M, N, K, group, t, relu in ((-1, 8, 8, 128, 0, 0), (8, -1, 8, 128, 0, 0), (8, 8, 2**31, 128, 0, 0),
                                    (65, 8, 8, 128, 0, 0), (8, 8, 8, 16, 0, 0), (8, 8, 8, 128, 2, 0), (8, 8, 8, 128, 0, 2)):
        assert L.linear_w4(16, t, 16, 16, None, 16, M, N, K, group, relu, None) == bad
    assert L.linear_w4(None, 0, 16, 16, None, 16, 8, 8, 8, 128, 0, None) == bad
    for t, st, trans in ((3, 0, 0), (0, 2, 0), (0, 0, 2)):
        assert L.w4_quantize(16, t, 16, 16, None, 8, 8, 128, st, trans, None) == bad
    assert L.w4_quantize(None, 0, 16, 16, None, 8, 8, 128, 0, 0, None) == bad


def test_empty_problems_are_no_ops_without_a_gpu(g):
    L = g.lib()
    for rows, dim in ((0, 8), (8, 0)):
        assert L.rms_norm_fwd(*[None] * 6, rows, dim, 0.0, 0, 0, None) == g.GEMM_OK
        assert L.rms_norm_fp8(*[None] * 7, rows, dim, 0.0, 0, 0, 0, None) == g.GEMM_OK
        assert L.rms_norm_bwd(*[None] * 7, rows, dim, 0, 0, None, 0, None) == g.GEMM_OK
        assert L.fp8_quantize(None, 0, None, None, rows, dim, 1, 0, None) == g.GEMM_OK
        assert L.w4_quantize(None, 0, None, None, None, rows, dim, 128, 0, 0, None) == g.GEMM_OK
        assert L.linear_w4(None, 0, None, None, None, None, rows, dim, 64, 128, 0, None) == g.GEMM_OK
    assert L.dropout_philox(None, None, None, 0, 0, 0.5, 0, 0, None, None) == g.GEMM_OK


def test_binding_refuses_wrong_tensors(g):
    x = torch.zeros((4, 128), dtype=H)
    w = torch.ones(128, dtype=H)
    r = torch.zeros(4)
    for call in (g.rms_norm_fwd, g.rms_norm_fp8, g.fp8_quantize, lambda t: g.dropout(t, 0.5, 0)):
        with pytest.raises(TypeError):
            call([1.0])
        for bad in (x.double(), x.t()):
            with pytest.raises(ValueError):
                call(bad)
    for call in (g.rms_norm_fwd, g.rms_norm_fp8):
        for kw in ({"gamma": w[:8]}, {"gamma": w.bfloat16()}, {"residual": x.float()}, {"residual": x[:2]}, {"H": x},
                   {"residual": x, "H": x.float()}):
            with pytest.raises(ValueError):
                call(x, **kw)
    with pytest.raises(ValueError):
        g.rms_norm_fp8(x, Q=x)
    with pytest.raises(ValueError):
        g.rms_norm_fp8(x, pow2=True, S=torch.zeros((4, 1)))
    for kw in ({"dY": x.float()}, {"rstd": r.half()}, {"dH": x[:2]}, {"wtype": torch.bfloat16}, {"dX": x.float()}):
        with pytest.raises(ValueError):
            g.rms_norm_bwd(**{"dY": x, "H": x, "rstd": r, **kw})
    with pytest.raises(ValueError):
        g.fp8_quantize(x, block_rows=64)
    for kw in ({"p": 1.0}, {"p": -0.1}, {"seed": -1}, {"offset": 2**64}, {"offset": r}, {"residual": x[:2]}, {"Y": x.float()}):
        with pytest.raises(ValueError):
            g.dropout(x, **{"p": 0.5, "seed": 0, **kw})
    Q, S, _ = g.w4_pack(torch.zeros((16, 128), dtype=U8), torch.zeros((16, 1), dtype=H))
    for args, kw in (((x.float(), Q, S), {}), ((x.bfloat16(), Q, S), {}), ((x, Q, S), {"group": 64}), ((x, Q, S), {"N": 17}),
                     ((x, Q, S, S), {}), ((x[:, :64].contiguous(), Q, S), {}), ((torch.zeros((65, 128), dtype=H), Q, S), {}),
                     ((x, Q, S), {"C": torch.zeros((4, 16))})):
        with pytest.raises(ValueError):
            g.linear_w4(*args, **kw)
    with pytest.raises(TypeError):
        g.linear_w4(x, [1], S)
    for args in ((torch.zeros((16, 128)), torch.zeros((16, 1), dtype=H)), (torch.zeros((16, 128), dtype=U8), torch.zeros((16, 1))),
                 (torch.zeros((16, 128), dtype=U8), torch.zeros((16, 2), dtype=H)),
                 (torch.zeros((16, 128), dtype=U8), torch.zeros((16, 1), dtype=H), torch.zeros((16, 1), dtype=H))):
        with pytest.raises(ValueError):
            g.w4_pack(*args)
    for kw in ({"group": 100}, {"stype": F}):
        with pytest.raises(ValueError):
            g.w4_quantize(x, **kw)


@pytest.mark.parametrize("N,K,group", [(1, 1, 128), (16, 64, 64), (37, 200, 32), (100, 129, 64)])
def test_packed_weights_have_the_documented_layout(g, N, K, group):
    gen = torch.Generator().manual_seed(N)
    q = torch.randint(0, 16, (N, K), generator=gen, dtype=U8)
    s = torch.randn((N, -(-K // group)), generator=gen).to(H)
    z = torch.randint(0, 16, s.shape, generator=gen, dtype=U8)
    Q, S, Z = g.w4_pack(q, s, z, group)
    assert (tuple(Q.shape), tuple(S.shape)) == g.w4_shapes(N, K, group) and S.shape == Z.shape
    assert torch.equal(ref.unpack_w4(Q, N, K), q.long())
    assert torch.equal(ref.per_column(S, N, K, group)[:, ::group], s.double())
    assert torch.equal(ref.weight_w4(Q, S, Z, N, K, group),
                       (q.double() - z.double().repeat_interleave(group, 1)[:, :K])
                       * s.double().repeat_interleave(group, 1)[:, :K])
    full = ref.unpack_w4(Q, 16 * Q.shape[0], 64 * Q.shape[1])
    assert (full[N:] == 0).all() and (full[:, K:] == 0).all()
