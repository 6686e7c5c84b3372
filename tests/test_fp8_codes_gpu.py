"""GPU tests of the last bit of E4M3 codes: quotients half way between two codes, and
blocks near the ends of binary32's range."""
from __future__ import annotations

import math

import pytest
import torch

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


def four_squares(n):
    """Four whole numbers whose squares add up to n."""
    for a in range(math.isqrt(n), -1, -1):
        for b in range(min(a, math.isqrt(n - a * a)), -1, -1):
            rest = n - a * a - b * b
            for c in range(min(b, math.isqrt(rest)), -1, -1):
                d = math.isqrt(rest - c * c)
                if d > c:
                    break
                if c * c + d * d == rest:
                    return [a, b, c, d]
    raise AssertionError(n)


def tie_rows(dim, dtype):
    """Rows of whole numbers, a block of 128 columns with a largest number a and another
    that is 448 y / a = half way between two E4M3 numbers, the others such that all
    squares add up to 2^23: the sum is exact in any order, and so is the norm's
    division, as dim is an odd power of 2."""
    rows = []
    for a in range(1, 129):
        ties = [n * 2.0 ** j * a / 448 for n in range(17, 32, 2) for j in range(-3, 5) if n * 2.0 ** j < 448]
        ties = [16 * y for y in ties if 16 * y == int(16 * y) and torch.tensor(16 * y).to(dtype).item() == 16 * y]
        for y in ties[:3] + ties[-3:]:
            rest = 2 ** 23 - (16 * a) ** 2 - int(y) ** 2
            row = torch.zeros(dim)
            row[0], row[5] = 16 * a, -y
            count = rest // 65536
            row[128:128 + count] = 256.0
            row[300:304] = torch.tensor(four_squares(rest - count * 65536)).float()
            assert float(row.double().square().sum()) == 2.0 ** 23
            rows.append(row)
    return torch.stack(rows)


@pytest.mark.parametrize("off_grid", [False, True])
@pytest.mark.parametrize("xt", list(DTYPES))
@pytest.mark.parametrize("dim", [512, 2048, 32768])
def test_norms_codes_half_way_between_two(g, dim, xt, off_grid):
    """The nearest code, and the even one of two as near, whatever the block's largest number."""
    h = tie_rows(dim, DTYPES[xt])
    rows = h.shape[0]
    assert rows > 100
    x = (h / 2).to(DTYPES[xt])
    assert torch.equal(x.double() * 2, h.double())
    flat = torch.empty(2 * rows * dim + 16, dtype=DTYPES[xt], device=DEV)
    at = 1 if off_grid else 0
    X, R = (flat[o:o + rows * dim].reshape(rows, dim) for o in (at, at + rows * dim + (8 if off_grid else 0)))
    X.copy_(x)
    R.copy_(x)
    Q, S, H = g.rms_norm_fp8(X, residual=R, eps=0.0)
    assert g.check() == g.GEMM_OK and torch.equal(H.double().cpu(), h.double())
    y = h.double() * (dim / 2.0 ** 23) ** 0.5
    assert torch.equal(S[:, 0].cpu(), (y[:, :128].abs().amax(1) / 448).float())
    want = (y[:, :128] * 448 / y[:, :128].abs().amax(1, keepdim=True)).float().to(torch.float8_e4m3fn)
    assert torch.equal(Q[:, :128].cpu().view(torch.uint8), want.view(torch.uint8))


@pytest.mark.parametrize("block_rows", [1, 128])
@pytest.mark.parametrize("exponent", [-149, -140, -131, -120, 80, 100])
def test_codes_of_blocks_near_the_ends_of_fp32(g, exponent, block_rows):
    """Whole numbers of up to 20 bits times a power of two, subnormals of few bits among them: the nearest codes."""
    gen = torch.Generator().manual_seed(exponent + 200)
    n = torch.randint(-2 ** 20, 2 ** 20, (64, 512), generator=gen).double()
    n *= torch.exp2(-torch.randint(0, 20, (64, 512), generator=gen).double())
    n[:8] = torch.randint(-5, 6, (8, 512), generator=gen).double()   # subnormals of three bits
    x = (n.round() * 2.0 ** exponent).float() + 0.0   # no -0
    Q, S = g.fp8_quantize(x.to(DEV), block_rows=block_rows)
    assert g.check() == g.GEMM_OK and torch.isfinite(S).all()
    b = x.double().reshape(64, 4, 128)
    a = b.abs().amax(2, keepdim=True)
    if block_rows == 128:
        a = a.amax(0, keepdim=True)
    assert (a > 0).all()
    v = (b * 448 / a).reshape(64, 512)
    want = v.float().to(torch.float8_e4m3fn)
    # The quotient is off by less than 2^-23, and exact half way between two codes.
    step = torch.exp2(torch.floor(torch.log2(v.abs().clamp(min=2.0 ** -6))) - 3)
    from_middle = ((v / step).abs() % 1 - 0.5).abs() * step
    clear = (from_middle == 0) | (from_middle > 2.0 ** -23 * v.abs())
    assert clear.double().mean() > 0.999
    assert torch.equal(Q.cpu().view(torch.uint8)[clear], want.view(torch.uint8)[clear])
