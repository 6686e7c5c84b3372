"""GPU tests of layer norm and its gradients against the formulas in 64 bits
and against differences."""
from __future__ import annotations

import pytest
import torch

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda:0")
DTYPES = {"fp16": torch.float16, "bf16": torch.bfloat16, "fp32": torch.float32}
TYPES = [("fp16", "fp16"), ("fp16", "fp32"), ("bf16", "bf16"), ("bf16", "fp32"), ("fp32", "fp32")]
# A thread adds up to 32 (long rows: 40) terms one by one, then a tree of 5 and
# up to 32 warps' sums: fewer than 96 roundings of 2^-24 each on any path.
U = 2.0 ** -24
ADDS = 96
EPS = 1e-5

SIZES = [(1, 1), (1, 7), (3, 8), (2, 255), (9, 256), (130, 264), (17, 512), (33, 513), (5, 1023), (300, 1024),
         (2, 1600), (700, 2048), (3, 4095), (64, 4096), (2, 4104), (400, 5000), (5, 8192), (3, 8200), (2, 16384),
         (2, 16385), (3, 32768), (2, 40000)]


@pytest.fixture(scope="module")
def g():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    from dense_fp16_gemm_05_gb300 import build as gbuild
    gbuild.build()
    from dense_fp16_gemm_05_gb300 import gemm_f16
    gemm_f16.lib()
    return gemm_f16


def half_step(t):
    """Half a step of type t relative to a value, and absolute near zero."""
    return torch.finfo(t).eps / 2, torch.finfo(t).smallest_normal * torch.finfo(t).eps


def draw(rows, dim, xt, wt, seed, shift=1.5):
    gen = torch.Generator().manual_seed(seed)
    x = (torch.randn((rows, dim), generator=gen) * 2 + shift * torch.randn((rows, 1), generator=gen)).to(xt)
    dy = torch.randn((rows, dim), generator=gen).to(xt)
    w = (1 + 0.3 * torch.randn(dim, generator=gen)).to(wt)
    b = (0.3 * torch.randn(dim, generator=gen)).to(wt)
    return [t.to(DEV) for t in (x, dy, w, b)]


def forward64(x, w, b):
    x = x.double()
    mean = x.mean(-1)
    z = x - mean[..., None]
    rstd = 1 / torch.sqrt((z * z).mean(-1) + EPS)
    z = z * rstd[..., None]
    y = z
    if w is not None:
        y = y * w.double()
    if b is not None:
        y = y + b.double()
    return y, mean, rstd, z


def check_forward(g, x, w, b):
    Y, mean, rstd = g.layer_norm_fwd(x, w, b, eps=EPS)
    Y2, none, none2 = g.layer_norm_fwd(x, w, b, eps=EPS, stats=False)
    assert g.check() == g.GEMM_OK and none is None and none2 is None
    assert torch.equal(Y, Y2)
    y, mu, r, z = forward64(x, w, b)
    A = x.double().abs().mean(-1)
    d_mu = (ADDS + 2) * U * A                       # the sum, the division
    d_r = ((ADDS + 8) / 2 * U + (d_mu * r) ** 2) * r   # half the variance's error
    assert ((mean.double() - mu).abs() <= d_mu + 1e-45).all()
    assert ((rstd.double() - r).abs() <= 1.01 * d_r + 2 * U * r).all()
    gw = 1.0 if w is None else w.double().abs()
    rel, tiny = half_step(x.dtype)
    d_z = (d_mu * r)[:, None] + z.abs() * (d_r / r + 4 * U)[:, None]
    tol = gw * d_z + 3 * U * (z.abs() * gw + y.abs()) + rel * y.abs() + tiny
    assert ((Y.double() - y).abs() <= 1.01 * tol).all()
    return mean, rstd


def check_backward(g, x, dy, w, mean, rstd, wt):
    dX, dg, db = g.layer_norm_bwd(dy, x, mean, rstd, w, wtype=wt if w is None else None)
    dX2, n1, n2 = g.layer_norm_bwd(dy, x, mean, rstd, w, weights=False)
    assert g.check() == g.GEMM_OK and n1 is None and n2 is None and torch.equal(dX, dX2)
    assert dg.dtype == wt and db.dtype == wt
    r, d = rstd.double()[:, None], dy.double()
    z = (x.double() - mean.double()[:, None]) * r
    gr = d if w is None else d * w.double()
    c1, c2 = gr.mean(-1, keepdim=True), (gr * z).mean(-1, keepdim=True)
    want = r * (gr - c1 - z * c2)
    d_z = 2 * U * (z.abs() + (mean.double().abs()[:, None]) * r)
    d_c1 = (ADDS + 3) * U * gr.abs().mean(-1, keepdim=True)
    d_c2 = (ADDS + 5) * U * (gr * z).abs().mean(-1, keepdim=True) + (gr.abs() * d_z).mean(-1, keepdim=True)
    rel, tiny = half_step(x.dtype)
    tol = r * (d_c1 + z.abs() * d_c2 + d_z * c2.abs() + 6 * U * (gr.abs() + c1.abs() + (z * c2).abs()))
    assert ((dX.double() - want).abs() <= 1.01 * (tol + rel * want.abs() + tiny)).all()
    rel, tiny = half_step(wt)
    for got, terms, err in ((dg, d * z, d.abs() * d_z), (db, d, torch.zeros_like(d))):
        s = terms.sum(0)
        # rows of a block one by one, then the blocks' sums
        tol = (ADDS + 3) * U * terms.abs().sum(0) + err.sum(0) + rel * s.abs() + tiny
        assert ((got.double() - s).abs() <= 1.01 * tol).all()
    return dX, dg, db


@pytest.mark.parametrize("xt,wt", TYPES)
@pytest.mark.parametrize("rows,dim", SIZES)
def test_forward_and_backward(g, rows, dim, xt, wt):
    x, dy, w, b = draw(rows, dim, DTYPES[xt], DTYPES[wt], rows * 31 + dim)
    mean, rstd = check_forward(g, x, w, b)
    check_backward(g, x, dy, w, mean, rstd, DTYPES[wt])


@pytest.mark.parametrize("xt,wt", TYPES)
@pytest.mark.parametrize("dim", [96, 1000, 2056])
def test_without_weights_and_with_one(g, dim, xt, wt):
    x, dy, w, b = draw(21, dim, DTYPES[xt], DTYPES[wt], dim)
    mean, rstd = check_forward(g, x, None, None)
    check_backward(g, x, dy, None, mean, rstd, DTYPES[wt])
    check_forward(g, x, w, None)
    check_forward(g, x, None, b)


@pytest.mark.parametrize("xt,wt", TYPES)
@pytest.mark.parametrize("dim", [64, 2048])
def test_unaligned_buffers_match_aligned_ones_within_rounding(g, dim, xt, wt):
    x, dy, w, b = draw(10, dim, DTYPES[xt], DTYPES[wt], 3)
    moved = []
    for t in (x, dy, w, b):
        flat = torch.empty(t.numel() + 1, dtype=t.dtype, device=DEV)
        flat[1:].copy_(t.reshape(-1))
        moved.append(flat[1:].reshape(t.shape))
    mean, rstd = check_forward(g, moved[0], moved[2], moved[3])
    check_backward(g, moved[0], moved[1], moved[2], mean, rstd, DTYPES[wt])


@pytest.mark.parametrize("rows,dim", [(5000, 128), (4097, 1030), (3000, 40)])
def test_more_rows_than_blocks(g, rows, dim):
    x, dy, w, b = draw(rows, dim, torch.float16, torch.float32, 7)
    mean, rstd = check_forward(g, x, w, b)
    first = check_backward(g, x, dy, w, mean, rstd, torch.float32)
    again = g.layer_norm_bwd(dy, x, mean, rstd, w)
    assert all(torch.equal(a, c) for a, c in zip(first, again))   # fixed order: the same bits


def test_large_mean_does_not_cancel(g):
    # deviations of 1/8 around 1000: sum x^2 - mean^2 would lose them in fp32
    x, _, w, b = draw(8, 1024, torch.float32, torch.float32, 1)
    x = 1000 + x / 16
    check_forward(g, x, w, b)


def test_constant_rows_and_special_values(g):
    x = torch.zeros((6, 256), dtype=torch.float16, device=DEV)
    x[0] = 3.0
    x[1, 5] = float("inf")
    x[2, 7] = float("nan")
    x[3] = torch.finfo(torch.float16).max
    b = torch.full((256,), 0.5, dtype=torch.float16, device=DEV)
    Y, mean, rstd = g.layer_norm_fwd(x, None, b, eps=EPS)
    assert (Y[[0, 3, 4, 5]] == 0.5).all()
    assert torch.isnan(Y[1]).any() and torch.isnan(Y[2]).all()
    assert mean[0] == 3.0 and mean[3] == 65504.0
    assert ((rstd[[0, 3, 4]].double() - EPS ** -0.5).abs() <= 4 * U * EPS ** -0.5 * 1.01 + 1e-6).all()


def test_leading_shapes_and_empty(g):
    x = torch.randn((2, 3, 5, 64), device=DEV)
    Y, mean, rstd = g.layer_norm_fwd(x)
    assert Y.shape == x.shape and mean.shape == (2, 3, 5)
    Y1, mean1, _ = g.layer_norm_fwd(x[0, 0, 0])
    assert mean1.shape == () and torch.equal(Y1, Y[0, 0, 0])
    e = torch.empty((0, 64), device=DEV)
    w = torch.ones(64, device=DEV)
    Y, mean, rstd = g.layer_norm_fwd(e, w, w)
    dX, dg, db = g.layer_norm_bwd(e, e, mean, rstd, w)
    assert dX.shape == (0, 64) and (dg == 0).all() and (db == 0).all()


def test_gradients_against_differences(g):
    from dense_fp16_gemm_05_gb300 import autograd as ag
    x, c, w, b = draw(3, 40, torch.float32, torch.float32, 12)
    leaves = [t.clone().requires_grad_() for t in (x, w, b)]
    (ag.layer_norm(*leaves, eps=EPS) * c).sum().backward()

    def f(x, w, b):
        return (forward64(x, w, b)[0] * c.double()).sum().item()

    args = [x.double(), w.double(), b.double()]
    h = 1e-4
    for which, leaf in enumerate(leaves):
        for idx in range(0, leaf.numel(), 7):
            lo, hi = [t.clone() for t in args], [t.clone() for t in args]
            lo[which].view(-1)[idx] -= h
            hi[which].view(-1)[idx] += h
            num = (f(*hi) - f(*lo)) / (2 * h)
            # the difference's own error is of order h^2 = 1e-8; fp32 sums of 40 terms below 1e-5
            assert abs(num - leaf.grad.view(-1)[idx].item()) <= 3e-5 * max(1.0, abs(num))


def test_autograd_partial_and_non_contiguous(g):
    from dense_fp16_gemm_05_gb300 import autograd as ag
    x = torch.randn((64, 48), device=DEV, dtype=torch.float16)
    w = torch.ones(64, device=DEV, dtype=torch.float16, requires_grad=True)
    y = ag.layer_norm(x.t(), w, None)           # non-contiguous input, no gradient for it
    y.sum().backward()
    want = forward64(x.t(), None, None)[3].sum(0)
    assert x.grad is None and torch.allclose(w.grad.double(), want, atol=2e-2)
    b = torch.zeros(64, device=DEV, dtype=torch.float32, requires_grad=True)
    xg = x.t().contiguous().requires_grad_()
    ag.layer_norm(xg, None, b).sum().backward()
    assert b.grad.dtype == torch.float32 and (b.grad == 48).all() and xg.grad.shape == xg.shape


def test_other_stream_and_graph_give_the_same_bits(g):
    x, dy, w, b = draw(50, 1024, torch.float16, torch.float16, 4)
    Y, mean, rstd = g.layer_norm_fwd(x, w, b)
    want = g.layer_norm_bwd(dy, x, mean, rstd, w)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = g.layer_norm_bwd(dy, x, mean, rstd, w, stream=side)
    side.synchronize()
    assert all(torch.equal(a, c) for a, c in zip(got, want))
    ws = torch.empty(g.layer_norm_bwd_workspace(50, 1024) // 4, device=DEV)
    graph = torch.cuda.CUDAGraph()
    y = torch.zeros_like(Y)
    with torch.cuda.graph(graph):
        _, m, r = g.layer_norm_fwd(x, w, b, Y=y)
        out = g.layer_norm_bwd(dy, x, m, r, w, workspace=ws)
    for _ in range(2):
        y.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, Y) and all(torch.equal(a, c) for a, c in zip(out, want))


def test_refusals(g):
    x = torch.zeros((4, 64), dtype=torch.float16, device=DEV)
    r = torch.zeros(4, device=DEV)
    L = g.lib()
    st = L.layer_norm_fwd(x.data_ptr(), None, None, x.data_ptr(), None, None, 4, 64, 0.0, 0, 0, None)
    assert st == g.GEMM_ERR_INVALID_ARG       # not in place
    with pytest.raises(g.GemmError):
        g.layer_norm_bwd(x, x, r, r, dX=x, weights=False)
    with pytest.raises(g.GemmError) as e:     # workspace too small
        g.layer_norm_bwd(x, x, r, r, workspace=torch.empty(16, device=DEV))
    assert e.value.status == g.GEMM_ERR_INVALID_ARG
    host = torch.zeros((4, 64), dtype=torch.float16)
    st = L.layer_norm_fwd(x.data_ptr(), None, None, host.data_ptr(), None, None, 4, 64, 0.0, 0, 0, None)
    assert st == g.GEMM_ERR_INVALID_ARG
    y = torch.empty_like(x)
    st = L.layer_norm_fwd(x.data_ptr() + 1, None, None, y.data_ptr(), None, None, 2, 64, 0.0, 0, 0, None)
    assert st == g.GEMM_ERR_ALIGNMENT
    st = L.layer_norm_fwd(x.data_ptr(), None, None, y.data_ptr(), None, None, 10**6, 64, 0.0, 0, 0, None)
    assert st == g.GEMM_ERR_INVALID_ARG       # past its allocation


@pytest.mark.parametrize("xt,wt", TYPES)
@pytest.mark.parametrize("rows,dim", [(3, 1500), (7, 2049), (2, 4099), (5, 6001)])
def test_operands_of_different_alignment(g, rows, dim, xt, wt):
    # X, dY and dX start at different places within 16 bytes, and dY ends with
    # its allocation
    x, dy, w, b = draw(rows, dim, DTYPES[xt], DTYPES[wt], rows + dim)
    moved = []
    for t, off in ((x, 1), (dy, 2)):
        flat = torch.empty(t.numel() + off, dtype=t.dtype, device=DEV)
        flat[off:].copy_(t.reshape(-1))
        moved.append(flat[off:].reshape(t.shape))
    guard = torch.full((rows * dim + 8,), 7.0, dtype=x.dtype, device=DEV)
    dX = guard[3:3 + rows * dim].reshape(rows, dim)
    mean, rstd = check_forward(g, moved[0], w, b)
    want, dg, db = check_backward(g, moved[0], moved[1], w, mean, rstd, DTYPES[wt])
    got, dg2, db2 = g.layer_norm_bwd(moved[1], moved[0], mean, rstd, w, dX=dX)
    assert got is dX and torch.equal(dX, want) and torch.equal(dg, dg2) and torch.equal(db, db2)
    assert (guard[:3] == 7.0).all() and (guard[3 + rows * dim:] == 7.0).all()
