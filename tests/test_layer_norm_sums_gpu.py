"""The column sums of the layer norm's backward pass where every block has one
row: what the blocks' parts lose when they are added is kept, so that the result
is the 64-bit sum rounded once."""
from __future__ import annotations

import pytest
import torch

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda:0")
U = 2.0 ** -24


@pytest.fixture(scope="module")
def g():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    from dense_fp16_gemm_05_gb300 import build as gbuild
    gbuild.build()
    from dense_fp16_gemm_05_gb300 import gemm_f16
    gemm_f16.lib()
    return gemm_f16


def check(got, terms):
    s, mag = terms.sum(0), terms.abs().sum(0)
    # one rounding of the result; the errors' own sum loses at most (n u)^2 of the magnitudes
    tol = U * s.abs() + (terms.shape[0] * U) ** 2 * mag
    assert ((got.double() - s).abs() <= 1.001 * tol).all()


# rows of the register, ring and long kernels, aligned and not
@pytest.mark.parametrize("rows,dim", [(300, 1024), (300, 1023), (300, 2500), (150, 6001), (150, 16384), (150, 16400),
                                      (7, 1024), (1, 1024)])
def test_parts_of_one_row_are_added_exactly(g, rows, dim):
    # Factors of 11 significant bits, mean 0 and rstd 1: every dy z is exact.
    gen = torch.Generator().manual_seed(rows + dim)
    x, dy = (torch.randn((rows, dim), generator=gen).half().float().to(DEV) for _ in range(2))
    mean, rstd = torch.zeros(rows, device=DEV), torch.ones(rows, device=DEV)
    _, dg, db = g.layer_norm_bwd(dy, x, mean, rstd, torch.ones(dim, device=DEV))
    assert g.check() == g.GEMM_OK
    check(dg, dy.double() * x.double())
    check(db, dy.double())


@pytest.mark.parametrize("over", [0, 1, 9])
def test_either_side_of_two_parts_per_sm(g, over):
    # a part per eight rows: where the second kernel's blocks change from 16 to 32 warps
    parts = 2 * torch.cuda.get_device_properties(DEV).multi_processor_count + over
    gen = torch.Generator(device=DEV).manual_seed(over)
    dy = torch.randint(-1000, 1001, (8 * parts, 768), generator=gen, device=DEV).float()   # sums exact in fp32
    x = torch.ones_like(dy)
    mean, rstd = torch.zeros(8 * parts, device=DEV), torch.ones(8 * parts, device=DEV)
    assert g.layer_norm_bwd_workspace(8 * parts, 768) == 8 * parts * 768
    _, dg, db = g.layer_norm_bwd(dy, x, mean, rstd)
    assert torch.equal(dg.double(), dy.double().sum(0)) and torch.equal(dg, db)


def test_sums_that_cancel(g):
    # 2^24 and its negative around small terms, which plain fp32 sums lose
    gen = torch.Generator().manual_seed(3)
    dy = torch.randn((200, 1024), generator=gen).half().float()
    dy[17], dy[120] = 2.0 ** 24, -2.0 ** 24
    dy = dy.to(DEV)
    x = torch.ones_like(dy)
    mean, rstd = torch.zeros(200, device=DEV), torch.ones(200, device=DEV)
    _, dg, db = g.layer_norm_bwd(dy, x, mean, rstd)
    check(dg, dy.double())
    check(db, dy.double())


@pytest.mark.parametrize("bad", [float("inf"), -float("inf"), float("nan")])
def test_infinities_stay_infinities(g, bad):
    dy = torch.ones((60, 1024), device=DEV)
    dy[11, 5] = bad
    x = torch.ones_like(dy)
    mean, rstd = torch.zeros(60, device=DEV), torch.ones(60, device=DEV)
    _, dg, db = g.layer_norm_bwd(dy, x, mean, rstd)
    for t in (dg, db):
        assert torch.isnan(t[5]) if bad != bad else t[5] == bad
        assert (t[:5] == 60).all() and (t[6:] == 60).all()
