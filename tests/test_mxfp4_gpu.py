"""GPU tests of MXFP4 quantisation and of the 4-bit product, against a plain
numpy restatement in 64 bits."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import mxfp4_reference as ref

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda:0")
DTYPES = {"fp16": torch.float16, "bf16": torch.bfloat16, "fp32": torch.float32}


@pytest.fixture(scope="module")
def g():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    from dense_fp16_gemm_05_gb300 import build as gbuild
    gbuild.build()
    from dense_fp16_gemm_05_gb300 import gemm_f16
    gemm_f16.lib()
    return gemm_f16


def draw(rows, K, dtype, seed):
    gen = torch.Generator().manual_seed(seed)
    x = torch.randn((rows, K), generator=gen) * torch.exp(2 * torch.randn((rows, 1), generator=gen))
    x = x.to(dtype)
    x[torch.rand((rows, K), generator=gen) < 0.05] = 0
    return x


def check_quantized(g, x, trans=False, offset=0):
    """Quantises x (rows, K) on the GPU and compares codes, scales and values, all exactly."""
    rows, K = x.shape
    src = (x.t() if trans else x).contiguous()
    if offset:   # a buffer that starts `offset` elements into its allocation
        flat = torch.empty(src.numel() + offset, dtype=src.dtype, device=DEV)
        dev = flat[offset:].reshape(src.shape)
        dev.copy_(src)
    else:
        dev = src.to(DEV)
    Q, S, V = g.mxfp4_quantize(dev, transpose=trans, values=True)
    Q2, S2 = g.mxfp4_quantize(dev, transpose=trans)
    assert g.check() == g.GEMM_OK
    KB = -(-K // 32)
    codes, scales = ref.quantize(x.double().numpy())
    got_s = ref.row_scales(S.cpu().numpy(), rows, 4 * S.shape[1])
    assert np.array_equal(got_s[:, :KB], scales)
    assert not got_s[:, KB:].any()
    assert np.array_equal(ref.decode(ref.unpack(Q.cpu().numpy()), np.full_like(scales, 127)),
                          ref.decode(codes, np.full_like(scales, 127)))
    # the values in X's type: one rounding of an exact product
    want = torch.from_numpy(ref.decode(codes, scales)[:, :K]).to(x.dtype)
    assert torch.equal(torch.nan_to_num(V.cpu().float(), nan=-7.0), torch.nan_to_num(want.float(), nan=-7.0))
    assert torch.equal(Q, Q2)
    got_s2 = ref.row_scales(S2.cpu().numpy(), rows, 4 * S.shape[1])
    assert np.array_equal(got_s, got_s2)


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("rows,K", [(1, 1), (1, 32), (3, 31), (2, 33), (5, 64), (33, 100), (130, 136), (1, 4096),
                                    (129, 264), (64, 250)])
@pytest.mark.parametrize("trans", [False, True])
def test_quantize(g, rows, K, dtype, trans):
    check_quantized(g, draw(rows, K, DTYPES[dtype], rows * 7 + K), trans)


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("trans", [False, True])
def test_quantize_unaligned_buffer(g, dtype, trans):
    check_quantized(g, draw(16, 64, DTYPES[dtype], 5), trans, offset=1)


@pytest.mark.parametrize("trans", [False, True])
@pytest.mark.parametrize("dtype", list(DTYPES))
def test_quantize_extremes(g, dtype, trans):
    t = DTYPES[dtype]
    info = torch.finfo(t)
    x = torch.zeros((8, 64), dtype=t)
    x[0, 0] = info.max
    x[1, 3], x[1, 4] = info.tiny, -info.tiny
    x[2, 5] = torch.finfo(t).smallest_normal * info.eps          # the smallest subnormal
    x[3, :32] = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 7.0] * 4, dtype=t)   # ties
    x[4, 7] = float("inf")
    x[5, 40] = float("nan")
    x[6, 2], x[6, 50] = -float("inf"), 3.0
    x[7, :] = -0.0
    check_quantized(g, x, trans)


def test_quantize_long_rows_and_many_rows(g):
    # more groups than the grid has threads, row ends inside a block of threads
    x = draw(1500, 2072, torch.float16, 3).to(DEV)
    Q, S, V = g.mxfp4_quantize(x, values=True)
    xt = x.t().contiguous()
    Qt, St, Vt = g.mxfp4_quantize(xt, transpose=True, values=True)
    assert g.check() == g.GEMM_OK
    rows = [0, 1, 127, 128, 1000, 1499]
    codes, scales = ref.quantize(x[rows].cpu().double().numpy())
    want = ref.decode(codes, scales)[:, :2072]
    assert np.array_equal(V[rows].cpu().double().numpy(), torch.from_numpy(want).half().double().numpy())
    assert torch.equal(Q, Qt) and torch.equal(V, Vt)
    KB = -(-2072 // 32)
    assert np.array_equal(ref.row_scales(S.cpu().numpy(), 1500, KB), ref.row_scales(St.cpu().numpy(), 1500, KB))


def operands(M, N, K, seed, lo=118, hi=128, fill=0):
    rng = np.random.default_rng(seed)
    out = []
    for rows in (M, N):
        KB = -(-K // 32)
        codes = rng.integers(0, 16, (rows, KB, 32), dtype=np.uint8)
        codes.reshape(rows, -1)[:, K:] = 0
        scales = rng.integers(lo, hi, (rows, KB), dtype=np.uint8)
        out.append((codes, scales))
    dev = []
    for codes, scales in out:
        dev += [torch.from_numpy(ref.pack(codes)).to(DEV), torch.from_numpy(ref.tile_scales(scales, fill)).to(DEV)]
    return out, dev


SIZES = [(1, 8, 32), (1, 8, 1), (7, 16, 33), (16, 136, 64), (31, 24, 250), (128, 128, 128), (129, 136, 160),
         (256, 256, 256), (64, 520, 513), (300, 520, 1000), (257, 264, 4095), (512, 768, 2048), (8, 2048, 4096),
         (1, 4096, 2080), (1000, 1000, 1000), (2, 8, 8192), (200, 3000, 96)]


@pytest.mark.parametrize("relu", [False, True])
@pytest.mark.parametrize("M,N,K", SIZES)
def test_product(g, M, N, K, relu):
    # rows past M and N of the scale tiles hold NaN scales, which no output may see
    (a, w), dev = operands(M, N, K, M + 3 * N + 7 * K, fill=255)
    C = torch.full((M + 2, N), 77.0, dtype=torch.float16, device=DEV)
    g.gemm_mxfp4(*dev, C=C[1:M + 1], relu=relu, K=K)
    assert g.check() == g.GEMM_OK
    got = C.cpu().double().numpy()
    assert np.all(got[0] == 77.0) and np.all(got[-1] == 77.0)   # nothing outside C
    want, mag = ref.product(ref.decode(*a)[:, :K], ref.decode(*w)[:, :K], relu)
    assert np.all(np.abs(got[1:-1] - want) <= ref.product_tolerance(want, mag, K))


@pytest.mark.parametrize("M,N,K", [(1, 64, 128), (40, 264, 640), (256, 512, 256), (300, 256, 1024)])
def test_product_exact_on_integers(g, M, N, K):
    # scales 2 and 4: every element is a whole number up to 24, every sum exact
    # in fp32, and the result is rounded once
    (a, w), dev = operands(M, N, K, 11, lo=128, hi=129)
    C = g.gemm_mxfp4(*dev, relu=False)
    assert g.check() == g.GEMM_OK
    want, _ = ref.product(ref.decode(*a), ref.decode(*w), False)
    assert torch.equal(C.cpu(), torch.from_numpy(want).half())


def test_product_sees_every_scale_in_its_place(g):
    # one nonzero element per row and block: the output is the product of two scales
    M, N, K = 256, 256, 512
    KB = K // 32
    rng = np.random.default_rng(2)
    for b in range(KB):
        codes = np.zeros((M, KB, 32), np.uint8)
        codes[:, b, (5 * b) % 32] = 2            # 1.0
        sa = rng.integers(120, 134, (M, KB), dtype=np.uint8)
        sw = rng.integers(120, 134, (N, KB), dtype=np.uint8)
        q = torch.from_numpy(ref.pack(codes)).to(DEV)
        C = g.gemm_mxfp4(q, torch.from_numpy(ref.tile_scales(sa)).to(DEV), q,
                         torch.from_numpy(ref.tile_scales(sw)).to(DEV))
        want = np.ldexp(1.0, sa[:, b].astype(int)[:, None] + sw[:, b].astype(int)[None, :] - 254)
        assert np.array_equal(C.cpu().double().numpy(), want), b


@pytest.mark.parametrize("M", [3, 300])
def test_nan_scale_reaches_its_row_only(g, M):
    (a, w), dev = operands(M, 64, 256, 4)
    x = torch.from_numpy(ref.decode(*a)).to(DEV).float()
    x[1, 40] = float("nan")
    Q, S = g.mxfp4_quantize(x)
    plain = g.gemm_mxfp4(Q, S, dev[2], dev[3], relu=False).cpu()
    relu = g.gemm_mxfp4(Q, S, dev[2], dev[3], relu=True).cpu()
    assert torch.isnan(plain[1]).all() and not torch.isnan(plain[[0, 2]]).any()
    assert (relu[1] == 0).all()


def test_empty_and_zero_k(g):
    C = torch.full((5, 16), 3.0, dtype=torch.float16, device=DEV)
    e = torch.empty(0, dtype=torch.uint8, device=DEV)
    g.gemm_mxfp4(e.reshape(5, 0), e.reshape(1, 0, 512), torch.empty((16, 0), dtype=torch.uint8, device=DEV),
                 e.reshape(1, 0, 512), C=C, K=0)
    assert (C == 0).all()
    Q, S = g.mxfp4_quantize(torch.empty((0, 64), dtype=torch.float16, device=DEV))
    assert Q.shape == (0, 32) and S.shape == (0, 1, 512)


@pytest.mark.parametrize("M", [4, 300])
def test_refusals(g, M):
    (_, _), dev = operands(M, 64, 96, 1)
    with pytest.raises(g.GemmError) as e:     # N % 8
        g.gemm_mxfp4(dev[0], dev[1], dev[2][:60], dev[3], K=96)
    assert e.value.status == g.GEMM_ERR_ALIGNMENT
    L = g.lib()
    C = torch.empty((M, 64), dtype=torch.float16, device=DEV)
    p = [t.data_ptr() for t in dev]
    assert L.gemm_mxfp4(p[0] + 8, p[1], p[2], p[3], C.data_ptr(), M, 64, 96, 0, None) == g.GEMM_ERR_ALIGNMENT
    assert L.gemm_mxfp4(p[0], p[1], p[2], p[3], p[0], M, 64, 96, 0, None) == g.GEMM_ERR_INVALID_ARG
    assert L.gemm_mxfp4(p[0], None, p[2], p[3], C.data_ptr(), M, 64, 96, 0, None) == g.GEMM_ERR_INVALID_ARG
    host = torch.empty((M, 64), dtype=torch.float16)
    assert L.gemm_mxfp4(p[0], p[1], p[2], p[3], host.data_ptr(), M, 64, 96, 0, None) == g.GEMM_ERR_INVALID_ARG
    X = torch.zeros((M, 96), dtype=torch.float16, device=DEV)
    assert L.mxfp4_quantize(X.data_ptr(), 0, X.data_ptr(), p[1], None, M, 96, 0, None) == g.GEMM_ERR_INVALID_ARG
    assert L.mxfp4_quantize(X.data_ptr(), 0, p[0], p[1], p[1], M, 96, 0, None) == g.GEMM_ERR_INVALID_ARG
    assert L.mxfp4_quantize(X.data_ptr() + 1, 0, p[0], p[1], None, M, 96, 0, None) == g.GEMM_ERR_ALIGNMENT


def test_other_stream_and_graph_give_the_same_bits(g):
    x = draw(40, 512, torch.float16, 9).to(DEV)
    (_, _), dev = operands(40, 256, 512, 8)
    Q, S = g.mxfp4_quantize(x)
    want = g.gemm_mxfp4(Q, S, dev[2], dev[3], relu=True)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        q, s = g.mxfp4_quantize(x)
        c = g.gemm_mxfp4(q, s, dev[2], dev[3], relu=True)
    side.synchronize()
    assert torch.equal(c, want)
    graph = torch.cuda.CUDAGraph()
    q, s, c = torch.zeros_like(Q), torch.zeros_like(S), torch.zeros_like(want)
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        g.mxfp4_quantize(x, Q=q, S=s)
        g.gemm_mxfp4(q, s, dev[2], dev[3], C=c, relu=True)
    for _ in range(3):
        c.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(c, want)


# 336, 288, 297, 256, 80 and 156 tiles: with and without half tiles at the end
@pytest.mark.parametrize("M,N,K", [(4096, 5128, 512), (3000, 6000, 260), (8200, 2056, 1100), (4096, 4096, 768),
                                   (2560, 2000, 512), (3012, 3304, 250)])
def test_product_more_tiles_than_sms(g, M, N, K):
    # several tiles per CTA pair: both accumulators and every ring slot in turn
    gen = torch.Generator(device=DEV).manual_seed(M)
    x = torch.randn((M, K), generator=gen, device=DEV, dtype=torch.bfloat16)
    w = torch.randn((N, K), generator=gen, device=DEV, dtype=torch.bfloat16)
    Q, S, V = g.mxfp4_quantize(x, values=True)
    Qw, Sw, Vw = g.mxfp4_quantize(w, values=True)      # values are exact in bf16
    C = g.gemm_mxfp4(Q, S, Qw, Sw, K=K)
    again = g.gemm_mxfp4(Q, S, Qw, Sw, K=K)
    assert g.check() == g.GEMM_OK
    assert torch.equal(C, again)
    want = V.double() @ Vw.double().t()
    mag = V.double().abs() @ Vw.double().abs().t()
    assert ((C.double() - want).abs() <= 2.0 ** -11 * want.abs() + 2.0 ** -25 + (K / 64 + 16) * 2.0 ** -22 * mag).all()


def test_calls_on_a_given_stream(g):
    # outputs made on the current stream, written on another: dropped at once,
    # their memory may not be handed out before the other stream is done
    x = draw(64, 4096, torch.float16, 2).to(DEV)
    (_, _), dev = operands(64, 256, 4096, 8)
    want_q, want_s = g.mxfp4_quantize(x)
    want = g.gemm_mxfp4(want_q, want_s, dev[2], dev[3])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    kept = []
    for i in range(20):
        q, s = g.mxfp4_quantize(x, stream=side)
        c = g.gemm_mxfp4(q, s, dev[2], dev[3], stream=side)
        kept.append(c)
        del q, s
        torch.full((64, 2048), i, dtype=torch.uint8, device=DEV)   # would land in q's memory
    side.synchronize()
    assert all(torch.equal(c, want) for c in kept)
