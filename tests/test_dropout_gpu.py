"""GPU tests of dropout: the mask bit for bit, values, streams of masks, graphs."""
from __future__ import annotations

import pytest
import torch

import feed_forward_reference as ref

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


def want(x, p, keep, r):
    """In fp32 with one rounding at the end: x / (1 - p) and the sum may each round once before."""
    y = torch.where(keep, x.double() * float(torch.tensor(1.0 / (1.0 - p), dtype=torch.float32)), 0.0)
    return y if r is None else y + r.double()


def check(x, p, keep, r, got):
    w = want(x, p, keep, r)
    # the product's and the sum's rounding in fp32, then the type's
    big = w.abs() if r is None else r.double().abs() + (w - r.double()).abs()
    tol = 2 * 2.0 ** -24 * big + torch.finfo(x.dtype).eps / 2 * w.abs() + torch.finfo(x.dtype).smallest_normal * 2.0 ** -11
    assert ((got.double() - w).abs() <= 1.01 * tol).all()
    if r is None:
        assert (got[~keep] == 0).all()
    else:
        assert torch.equal(got[~keep], r[~keep])


@pytest.mark.parametrize("xt", list(DTYPES))
@pytest.mark.parametrize("n", [1, 3, 4, 5, 8, 9, 255, 1021, 4096])
@pytest.mark.parametrize("residual", [False, True])
def test_mask_and_values(g, n, xt, residual):
    gen = torch.Generator().manual_seed(n)
    x, r = ((1 + torch.rand(n, generator=gen)).to(DTYPES[xt]).to(DEV) for _ in range(2))
    r = r if residual else None
    for p, seed, offset in ((0.1, 1, 0), (0.5, 2 ** 64 - 1, 2 ** 64 - 2), (0.25, 0x123456789ABCDEF0, 2 ** 32)):
        y = g.dropout(x, p, seed, offset, residual=r)
        assert g.check() == g.GEMM_OK
        check(x, p, ref.kept(0, n, p, seed, offset).to(DEV), r, y)


def test_unaligned_views_and_in_place(g):
    gen = torch.Generator().manual_seed(1)
    for t in DTYPES.values():
        base = torch.randn(2049, generator=gen).to(t).to(DEV)
        x = base[1:]
        r = torch.randn(2048, generator=gen).to(t).to(DEV)
        keep = ref.kept(0, 2048, 0.3, 9, 4).to(DEV)
        for a in (x, x.clone()):
            y = g.dropout(a, 0.3, 9, 4, residual=r)
            check(a, 0.3, keep, r, y)
            b, c = a.clone(), r.clone()
            assert torch.equal(g.dropout(b, 0.3, 9, 4, residual=c, Y=c), y) and torch.equal(b, a)
            assert torch.equal(g.dropout(b, 0.3, 9, 4, residual=r, Y=b), y) and torch.equal(b, y)
    assert g.check() == g.GEMM_OK


def test_infinities_and_nan_are_dropped_too(g):
    x = torch.full((4096,), float("inf"), device=DEV).half()
    x[::2] = float("nan")
    y = g.dropout(x, 0.5, 3)
    keep = ref.kept(0, 4096, 0.5, 3, 0).to(DEV)
    assert (y[~keep] == 0).all() and torch.equal(torch.isnan(y), keep & torch.isnan(x))


def test_probability_zero_keeps_everything(g):
    x = torch.randn(1000, device=DEV)
    assert torch.equal(g.dropout(x, 0.0, 5), x)
    r = torch.randn(1000, device=DEV)
    assert torch.equal(g.dropout(x, 0.0, 5, residual=r), x + r)


@pytest.mark.parametrize("p", [0.001, 0.1, 0.5, 0.9])
def test_share_of_kept_elements(g, p):
    n = 1 << 22
    x = torch.ones(n, device=DEV)
    masks = [g.dropout(x, p, 7, o) != 0 for o in range(2)] + [g.dropout(x, p, 8, 0) != 0]
    sd = (p * (1 - p) / n) ** 0.5
    for m in masks:
        assert abs(m.double().mean().item() - (1 - p)) <= 5 * sd
    # masks of other offsets and seeds agree as independent ones do
    for i, j in ((0, 1), (0, 2), (1, 2)):
        both = (masks[i] & masks[j]).double().mean().item()
        q = (1 - p) ** 2
        assert abs(both - q) <= 5 * (q * (1 - q) / n) ** 0.5


def test_offset_in_device_memory(g):
    x = torch.randn((33, 77), device=DEV).half()
    for o in (0, 5, 2 ** 40 + 3):
        off = torch.tensor([o], device=DEV)
        assert torch.equal(g.dropout(x, 0.2, 11, off), g.dropout(x, 0.2, 11, o))


def test_captured_graph_draws_another_mask_at_every_replay(g):
    x = torch.randn((64, 128), device=DEV).half()
    off = torch.zeros(1, dtype=torch.int64, device=DEV)
    y = torch.empty_like(x)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        g.dropout(x, 0.5, 21, off, Y=y)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        g.dropout(x, 0.5, 21, off, Y=y)
        off.add_(1)
    for i in range(3):
        graph.replay()
        torch.cuda.synchronize()
        assert int(off) == i + 1
        assert torch.equal(y, g.dropout(x, 0.5, 21, i))


def test_more_elements_than_32_bits_count(g):
    n = (1 << 32) + 1029
    x = torch.ones(n, dtype=torch.float16, device=DEV)
    g.dropout(x, 0.5, 3, 1, Y=x)
    for first in (0, (1 << 31) - 8, (1 << 32) - 8, n - 1000):
        m = min(1000, n - first)
        assert torch.equal(x[first:first + m].cpu() != 0, ref.kept(first, m, 0.5, 3, 1))
    del x
    torch.cuda.empty_cache()


def test_refusals(g):
    x = torch.zeros(64, device=DEV).half()
    for p in (-0.1, 1.0, 2.0, float("nan")):
        with pytest.raises(ValueError):
            g.dropout(x, p, 0)
    for seed, offset in ((-1, 0), (1 << 64, 0), (0, -1), (0, 1 << 64)):
        with pytest.raises(ValueError):
            g.dropout(x, 0.5, seed, offset)
    for off in (torch.zeros(1, device=DEV), torch.zeros(2, dtype=torch.int64, device=DEV),
                torch.zeros(1, dtype=torch.int64)):
        with pytest.raises(ValueError):
            g.dropout(x, 0.5, 0, off)
    with pytest.raises(ValueError):
        g.dropout(x, 0.5, 0, residual=x.float())
    buf = torch.zeros(72, device=DEV).half()
    with pytest.raises(g.GemmError):
        g.dropout(buf[:64], 0.5, 0, Y=buf[8:])
    assert g.dropout(x[:0], 0.5, 0).numel() == 0
