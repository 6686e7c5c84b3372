"""GPU tests of the RMS norm of rows whose squares vanish in binary32, with an eps that
does not hide them."""
from __future__ import annotations

import pytest
import torch

import feed_forward_reference as ref
from test_rms_norm_gpu import ADDS, D_R, DEV, DTYPES, U, check_backward, g, half_step  # noqa: F401  (g: a fixture)

pytestmark = pytest.mark.gpu

# In turn, so that a warp of short rows has some of each.
SCALES = [1.0, 1e-19, 1e-20, 1e-16, 1e-25, 1e-30, 1e-38, 3e-40, 1e19, 1e-12]


@pytest.mark.parametrize("eps", [0.0, 1e-44, 1e-36])
@pytest.mark.parametrize("xt", ["bf16", "fp32"])
@pytest.mark.parametrize("dim", [8, 40, 100, 512, 1001, 4096, 4097, 8200, 20001])
def test_rows_whose_squares_vanish(g, dim, xt, eps):  # noqa: F811
    gen = torch.Generator().manual_seed(dim)
    rows = 1300 if dim == 4097 else 30   # the kernel for many shifted rows
    scale = torch.tensor(SCALES, dtype=torch.float64).repeat(rows // 10).reshape(-1, 1)
    x = (torch.randn((rows, dim), generator=gen).double().clamp(-4, 4) * scale).to(DTYPES[xt]).to(DEV)
    r = (x.double() / 3).to(x.dtype)
    rel, tiny = half_step(x.dtype)
    for residual in (None, r):
        Y, H, rstd = g.rms_norm_fwd(x, residual=residual, eps=eps)
        h = H.double()
        e = float(torch.tensor(eps, dtype=torch.float32))
        want = 1 / torch.sqrt((h * h).mean(-1) + e)
        largest = torch.finfo(torch.float32).max
        inside = want < 0.9 * largest
        # beyond binary32 (a root mean square below 2^-128): infinite
        assert ((rstd.double() - want).abs() <= D_R * want + 2.0 ** -149)[inside].all()
        assert torch.isinf(rstd[want > 1.1 * largest]).all()
        y = h * want[:, None]
        # rstd below 2^-126 has steps of 2^-149
        d = (D_R + 2.0 ** -149 / want + 3 * U)[:, None]
        assert ((Y.double() - y).abs() <= (d + rel) * 1.001 * y.abs() + tiny)[inside].all()
        Q, S, _ = g.rms_norm_fp8(x, residual=residual, eps=eps)
        v = Q.float().double() * ref.spread(S.double(), 1, rows, dim)
        a = ref.spread(ref.blocks(y, 1).abs().amax(dim=(1, 3)), 1, rows, dim)
        assert ((v - y).abs() <= 2.0 ** -4 * 1.001 * y.abs() + a * 2.0 ** -17)[inside].all()
    assert g.check() == g.GEMM_OK


@pytest.mark.parametrize("dim", [96, 2048, 2049])
@pytest.mark.parametrize("scale", [1e-20, 1e-30])
def test_gradients_of_such_rows(g, dim, scale):  # noqa: F811
    gen = torch.Generator().manual_seed(dim)
    x, dy = (torch.randn((5, dim), generator=gen).to(DEV) for _ in range(2))
    x = x * scale
    w = (1 + 0.3 * torch.randn(dim, generator=gen)).to(DEV)
    _, H, rstd = g.rms_norm_fwd(x, w, eps=0.0)
    check_backward(g, H, dy, w, rstd, torch.float32, None)


def test_rows_of_zeros_are_what_the_formula_gives(g):  # noqa: F811
    x = torch.zeros((3, 256), device=DEV)
    x[1] = 1e-30
    Y, _, rstd = g.rms_norm_fwd(x, eps=0.0)
    assert torch.isinf(rstd[[0, 2]]).all() and torch.isnan(Y[[0, 2]]).all()
    assert ((Y[1] - 1).abs() < 2.0 ** -20).all()
    Y, _, rstd = g.rms_norm_fwd(x, eps=1e-30)
    assert (Y[0] == 0).all() and torch.isfinite(Y).all()
