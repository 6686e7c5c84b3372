"""GPU tests of the FP8 block quantisation against the definition in 64 bits."""
from __future__ import annotations

import pytest
import torch

import feed_forward_reference as ref

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda:0")
DTYPES = {"fp16": torch.float16, "bf16": torch.bfloat16, "fp32": torch.float32}
U = 2.0 ** -24
SIZES = [(1, 1), (1, 8), (3, 127), (5, 128), (2, 129), (130, 136), (256, 256), (7, 1000), (33, 1001), (257, 2056),
         (64, 8192), (1000, 392), (129, 640)]


@pytest.fixture(scope="module")
def g():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    from dense_fp16_gemm_05_gb300 import build as gbuild
    gbuild.build()
    from dense_fp16_gemm_05_gb300 import gemm_f16
    gemm_f16.lib()
    return gemm_f16


def check(g, x, block_rows, pow2):
    Q, S = g.fp8_quantize(x, block_rows=block_rows, pow2=pow2)
    assert g.check() == g.GEMM_OK
    rows, K = x.shape
    xd = x.double()
    a = ref.blocks(xd, block_rows).abs().amax(dim=(1, 3))
    assert Q.dtype == torch.float8_e4m3fn and S.shape == a.shape
    # A value beyond the type (the wide draw below has some in fp16) is an infinity:
    # its block is NaN in scale and codes.  The others are held to the definition.
    beyond = ~torch.isfinite(a)
    assert torch.equal(S == 255 if pow2 else torch.isnan(S), beyond)
    lost = ref.spread(beyond, block_rows, rows, K)
    assert torch.isnan(Q.float())[lost].all()
    xd = torch.where(lost, 0.0, xd)
    a = torch.where(beyond, 0.0, a)
    S = torch.where(beyond, torch.full_like(S, 127 if pow2 else 1), S)
    if pow2:
        # The least power of two that keeps the block's values at or below 448, no less than 2^-127.
        s = torch.exp2(S.double() - 127)
        assert (a <= 448 * s).all()
        assert ((a > 224 * s) | (S == 0) | ((a == 0) & (S == 127))).all()
    else:
        # Rounded once (in 32 bits torch multiplies by 1 / 448, which rounds twice; the
        # 53-bit quotient of a 24-bit number by 7 2^6 is never half way between two).
        want = torch.where(a > 0, a / 448, torch.ones_like(a)).float()
        assert torch.equal(S, want)
        s = torch.where(a > 0, a / 448, torch.ones_like(a))
    sv = ref.spread(s, block_rows, rows, K)
    # Without the scale's rounding: 448 x / a keeps ties, and s x in 64 bits is exact to 2^-53.
    v = xd / sv if pow2 else xd * 448 / ref.spread(torch.where(a > 0, a, 448 * torch.ones_like(a)), block_rows, rows, K)
    err = 0.0 if pow2 else 2 * U * v.abs()   # the quotient's rounding; none of 448 x in 16-bit types
    got = torch.where(lost, 0.0, Q.float().double())
    assert ((got - v).abs() <= ref.e4m3_half_step(v.abs()) + err).all()
    # Ties and everything else off the midpoints' neighbourhood: the nearest code itself.
    nearest = v.float().clamp(-448, 448).to(torch.float8_e4m3fn).float().double()
    clear = ((v - nearest).abs() - ref.e4m3_half_step(v)).abs() > 4 * U * v.abs()
    if x.dtype != torch.float32 or pow2:
        clear |= v == v.float().double()   # representable quotients, ties among them
    assert torch.equal(got[clear], nearest[clear])


@pytest.mark.parametrize("pow2", [False, True])
@pytest.mark.parametrize("block_rows", [1, 128])
@pytest.mark.parametrize("xt", list(DTYPES))
@pytest.mark.parametrize("rows,K", SIZES)
def test_quantisation(g, rows, K, xt, block_rows, pow2):
    gen = torch.Generator().manual_seed(rows * 7 + K)
    x = torch.randn((rows, K), generator=gen) * torch.exp(3 * torch.randn((1, K), generator=gen))
    x[torch.rand((rows, K), generator=gen) < 0.05] = 0.0
    if rows > 2:
        x[1] = 0.0
    check(g, x.to(DTYPES[xt]).to(DEV), block_rows, pow2)


@pytest.mark.parametrize("pow2", [False, True])
@pytest.mark.parametrize("xt", list(DTYPES))
def test_unaligned_and_strided_views(g, xt, pow2):
    gen = torch.Generator().manual_seed(3)
    x = torch.randn((40, 256), generator=gen).to(DTYPES[xt]).to(DEV)
    flat = torch.empty(x.numel() + 1, dtype=x.dtype, device=DEV)
    flat[1:].copy_(x.reshape(-1))
    view = flat[1:].reshape(40, 256)
    for block_rows in (1, 128):
        want, got = g.fp8_quantize(x, block_rows, pow2), g.fp8_quantize(view, block_rows, pow2)
        Q = torch.empty(40 * 256 + 3, dtype=torch.uint8, device=DEV)[3:].view(torch.float8_e4m3fn).reshape(40, 256)
        off = g.fp8_quantize(x, block_rows, pow2, Q=Q)
        for o in (got, off):
            assert torch.equal(o[0].view(torch.uint8), want[0].view(torch.uint8)) and torch.equal(o[1], want[1])
    with pytest.raises(ValueError):
        g.fp8_quantize(x.t())


@pytest.mark.parametrize("pow2", [False, True])
@pytest.mark.parametrize("scale", [1e-44, 1e-40, 1e-38, 3e-36, 1e-33, 1e30, 1e35, 3e38])
def test_the_ends_of_fp32(g, scale, pow2):
    x = (torch.linspace(-1, 1, 256, dtype=torch.float64).reshape(2, 128) * scale).float().to(DEV)
    Q, S = g.fp8_quantize(x, pow2=pow2)
    assert torch.isfinite(Q.float()).all()
    if pow2:
        # below 2^-127 448 the least scale, codes as they come
        s = torch.exp2(S.double() - 127)
        assert (x.double().abs().amax(1, keepdim=True) <= 448 * s).all()
        v = x.double() / s
    else:
        assert torch.isfinite(S).all()
        v = x.double() * 448 / x.double().abs().amax(1, keepdim=True)
    # 7/8 x of a subnormal x is rounded to a step of 2^-149
    err = 4 * U * v.abs() + (0 if pow2 else 2.0 ** -149 * 512 / x.double().abs().amax(1, keepdim=True))
    assert ((Q.float().double() - v).abs() <= ref.e4m3_half_step(v.abs()) + err).all()


@pytest.mark.parametrize("block_rows", [1, 128])
@pytest.mark.parametrize("K", [128, 300, 301])
def test_infinities_and_nan_are_not_hidden(g, K, block_rows):
    x = torch.randn((130, K), device=DEV).half()
    x[0, K - 1] = float("nan")
    x[129, 0] = -float("inf")
    Q, S = g.fp8_quantize(x, block_rows)
    last = (K - 1) // 128
    assert torch.isnan(S[0, last]) and torch.isnan(S[-1, 0]) and int(torch.isnan(S).sum()) == 2
    assert torch.isnan(Q[0, last * 128:].float()).all() and torch.isnan(Q[129, :128].float()).all()
    _, S = g.fp8_quantize(x, block_rows, pow2=True)
    assert S[0, last] == 255 and S[-1, 0] == 255 and int((S == 255).sum()) == 2


def test_empty_and_refused(g):
    e = torch.empty((0, 64), device=DEV).half()
    Q, S = g.fp8_quantize(e)
    assert Q.shape == (0, 64) and S.shape == (0, 1)
    x = torch.zeros((4, 64), device=DEV).half()
    with pytest.raises(ValueError):
        g.fp8_quantize(x, block_rows=2)
    with pytest.raises(ValueError):
        g.fp8_quantize(x, S=torch.empty((4, 1), dtype=torch.uint8, device=DEV))
    with pytest.raises(g.GemmError):
        g.fp8_quantize(x, Q=x.view(torch.float8_e4m3fn).reshape(-1)[:256].reshape(4, 64))


@pytest.mark.parametrize("pow2", [False, True])
def test_products_take_the_quantised_operands(g, pow2):
    """The product of a norm's FP8 output with an FP8 weight is the product of what the codes stand for."""
    gen = torch.Generator().manual_seed(5)
    x, r = (torch.randn((70, 512), generator=gen).half().to(DEV) for _ in range(2))
    w = (torch.randn((264, 512), generator=gen) / 512 ** 0.5).half().to(DEV)
    A, SA, H = g.rms_norm_fp8(x, residual=r, pow2=pow2)
    W, SW = g.fp8_quantize(w, block_rows=128, pow2=pow2)
    C = (g.gemm_mxfp8_block_scaled if pow2 else g.gemm_fp8_block_scaled)(A, SA, W, SW, relu=False)
    assert g.check() == g.GEMM_OK
    sa, sw = (torch.exp2(s.double() - 127) if pow2 else s.double() for s in (SA, SW))
    av = A.float().double() * ref.spread(sa, 1, 70, 512)
    wv = W.float().double() * ref.spread(sw, 128, 264, 512)
    want = av @ wv.t()
    # 512 products in fp32, in any order, and one rounding to fp16
    tol = 512 * 2 * U * (av.abs() @ wv.abs().t()) + 2.0 ** -11 * want.abs() + 2.0 ** -25
    assert ((C.double() - want).abs() <= tol).all()
