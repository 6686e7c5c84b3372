"""Offsets past 2^31 elements, codes past 4 GiB and the widest rows in the operators around
a feed-forward block: against the same rows in small calls, or against 64 bits."""
from __future__ import annotations

import pytest
import torch

import feed_forward_reference as ref
from test_feed_forward_sizes_gpu import big_rows, release  # noqa: F401  (release: a fixture of every test)

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda:0")
U = 2.0 ** -24
REL = torch.finfo(torch.bfloat16).eps / 2   # a rounding to bf16: 2^-8


@pytest.fixture(scope="module")
def g():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    from dense_fp16_gemm_05_gb300 import build as gbuild
    gbuild.build()
    from dense_fp16_gemm_05_gb300 import gemm_f16
    gemm_f16.lib()
    return gemm_f16


def spots(rows, n):
    """The first rows, some at 2^31 elements' half and the last ones, from multiples of 128 on."""
    return [(a, min(a + n, rows)) for a in (0, rows // 256 * 128, (rows - n) // 128 * 128 + 128)]


# A row per block, per shifted block, element by element, per warp, and of no block's size.
@pytest.mark.parametrize("dim", [16384, 4097, 520, 515, 32776])
def test_norm_past_2_31_elements(g, dim):
    rows = (2 ** 31 + 2 ** 26) // dim // 128 * 128 + 72
    n = max(256, (1 << 22) // dim // 128 * 128 + 256)   # as many as the shifted kernel asks for
    x = big_rows(rows, dim, torch.float16)
    r = x.flip(0)
    w = torch.linspace(0.5, 1.5, dim, device=DEV).half()
    Y, H, rstd = g.rms_norm_fwd(x, w, residual=r)
    assert x.numel() > 2 ** 31
    for a, b in spots(rows, n):
        y, h, s = g.rms_norm_fwd(x[a:b].clone(), w, residual=r[a:b].clone())
        assert torch.equal(Y[a:b], y) and torch.equal(H[a:b], h) and torch.equal(rstd[a:b], s)
    Q, S, _ = g.rms_norm_fp8(x, w, residual=r, H=r)
    for a, b in spots(rows, n):
        q, s, _ = g.rms_norm_fp8(H[a:b].clone(), w)
        assert torch.equal(Q[a:b].view(torch.uint8), q.view(torch.uint8)) and torch.equal(S[a:b], s)
    del Q, S
    assert torch.equal(r, H)
    dX, dg = g.rms_norm_bwd(Y, H, rstd, w, dH=x)
    assert g.check() == g.GEMM_OK
    for a, b in spots(rows, n):
        y, h, s = Y[a:b].double(), H[a:b].double(), rstd[a:b].double()[:, None]
        z, gr = h * s, y * w.double()
        want = x[a:b].double() + s * (gr - z * (gr * z).mean(1, keepdim=True))
        # a row's sum in at most dim / 1024 + 16 roundings, then some of a few terms
        tol = s * z.abs() * (dim / 1024 + 24) * U * (gr * z).abs().mean(1, keepdim=True) + 8 * U * (s * gr.abs() + want.abs())
        assert ((dX[a:b].double() - want).abs() <= 1.01 * (tol + 2.0 ** -11 * want.abs() + 2.0 ** -25)).all()
    want = torch.zeros(dim, dtype=torch.float64, device=DEV)
    mag = torch.zeros_like(want)
    step = (1 << 27) // dim
    for a in range(0, rows, step):
        t = Y[a:a + step].double() * H[a:a + step].double() * rstd[a:a + step].double()[:, None]
        want += t.sum(0)
        mag += t.abs().sum(0)
    # at most rows / 152 + 8 terms one by one, then the blocks' sums
    tol = (rows / 152 + 24) * U * mag + 2.0 ** -11 * want.abs() + 2.0 ** -24
    over = want.abs() - tol > 65520
    sure = (want.abs() + tol < 65520) | over
    assert torch.equal(torch.isinf(dg) & sure, over)
    assert ((dg.double() - want).abs() <= 1.01 * tol)[sure & ~over].all()


@pytest.mark.parametrize("pow2", [False, True])
@pytest.mark.parametrize("dim", [32776, 32771])
def test_fp8_codes_past_2_31_elements(g, dim, pow2):
    rows = 66000
    x = big_rows(rows, dim, torch.bfloat16)
    for block_rows in (1, 128):
        Q, S = g.fp8_quantize(x, block_rows, pow2)
        assert g.check() == g.GEMM_OK
        for a, b in spots(rows, 256):
            q, s = g.fp8_quantize(x[a:b].clone(), block_rows, pow2)
            assert torch.equal(Q[a:b].view(torch.uint8), q.view(torch.uint8))
            assert torch.equal(S[a // block_rows:-(-b // block_rows)], s)


def test_weight_of_more_than_4_gib_of_codes(g):
    N, K, group = 2 ** 20 + 24, 8328, 128
    w = big_rows(N, K, torch.float16)
    W = g.w4_quantize(w, group, zeros=True)
    assert g.check() == g.GEMM_OK and W[0].numel() > 2 ** 32
    for a, b in [(0, 128), (N // 2 // 16 * 16, N // 2 // 16 * 16 + 64), (N // 16 * 16 - 64, N)]:
        part = g.w4_quantize(w[a:b].clone(), group, zeros=True)
        for whole, p in zip(W, part):
            assert torch.equal(whole[a // 16:-(-b // 16)], p)
    del w
    gen = torch.Generator().manual_seed(5)
    for M in (1, 8, 16, 30, 64):
        X = torch.randn((M, K), generator=gen).half().to(DEV)
        C = g.linear_w4(X, *W, N=N, group=group)
        assert g.check() == g.GEMM_OK
        for a, b in [(0, 256), (N // 2 // 16 * 16, N // 2 // 16 * 16 + 64), (N // 16 * 16 - 256, N)]:
            part = [t[a // 16:-(-b // 16)] for t in W]
            v = ref.weight_w4(*part, b - a, K, group)
            want = X.double() @ v.t()
            # as for any size: a group's eight products, the groups', warps' and blocks' sums
            steps = 2 * 17 * 8 + 2 * (K // 128 + 1) + 80
            tol = steps * U * (X.double().abs() @ v.abs().t()) + 2.0 ** -11 * want.abs() + 2.0 ** -25
            assert ((C[:, a:b].double() - want).abs() <= 1.01 * tol).all()


@pytest.mark.parametrize("dim", [2 ** 31 - 1, 2 ** 31 - 7, 2 ** 31 - 8])
def test_the_widest_row(g, dim):
    """Whole numbers of -2 .. 2, whose sums are exact in binary32 but for the last tree."""
    x = torch.randint(-2, 3, (1, dim), dtype=torch.int8, device=DEV).bfloat16()
    Y, H, rstd = g.rms_norm_fwd(x, eps=0.0)
    assert g.check() == g.GEMM_OK
    mean = sum(float(x[0, a:a + 2 ** 28].double().square().sum()) for a in range(0, dim, 2 ** 28)) / dim
    # a tree of ten additions, the mean, the root and the division
    assert abs(float(rstd) * mean ** 0.5 - 1) <= 16 * U
    for a in (0, dim // 2, dim - 4096):
        y = x[0, a:a + 4096].double() / mean ** 0.5
        assert ((Y[0, a:a + 4096].double() - y).abs() <= (REL + 20 * U) * y.abs()).all()
    Q, S, _ = g.rms_norm_fp8(x, eps=0.0)
    for a in (0, dim // 2 // 128 * 128, (dim - 4096) // 128 * 128):
        part = slice(a, a + 4096)
        q = Q[0, part].float().double()
        v = q * S[0, a // 128:a // 128 + 32].repeat_interleave(128).double()[:q.numel()]
        y = x[0, part].double() / mean ** 0.5
        assert ((v - y).abs() <= 2.0 ** -4 * 1.001 * y.abs()).all()
    del Q, S, Y
    dy = torch.randint(-2, 3, (1, dim), dtype=torch.int8, device=DEV).bfloat16()
    half = torch.full((1,), 0.5, device=DEV)
    dX, dg = g.rms_norm_bwd(dy, x, half)
    assert g.check() == g.GEMM_OK
    c = sum(float((dy[0, a:a + 2 ** 28].double() * x[0, a:a + 2 ** 28].double()).sum()) for a in range(0, dim, 2 ** 28)) * 0.5 / dim
    for a in (0, dim // 2, dim - 4096):
        d, h = dy[0, a:a + 4096].double(), x[0, a:a + 4096].double()
        want = 0.5 * (d - 0.5 * h * c)
        assert ((dX[0, a:a + 4096].double() - want).abs() <= (REL + 4 * U) * want.abs() + 16 * U * (h * c).abs() + 2.0 ** -30).all()
        assert torch.equal(dg[a:a + 4096].double(), 0.5 * d * h)
