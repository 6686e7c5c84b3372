"""GPU tests of the RMS norm, its FP8 output and its gradients against the
formulas in 64 bits and against differences."""
from __future__ import annotations

import pytest
import torch

import feed_forward_reference as ref

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda:0")
DTYPES = {"fp16": torch.float16, "bf16": torch.bfloat16, "fp32": torch.float32}
TYPES = [("fp16", "fp16"), ("fp16", "fp32"), ("bf16", "bf16"), ("bf16", "fp32"), ("fp32", "fp32")]
# A thread adds up to 32 (long rows: 40) terms one by one, then a tree of 5 and
# up to 32 warps' sums: fewer than 96 roundings of 2^-24 each on any path.
U = 2.0 ** -24
ADDS = 96
EPS = 1e-6
# The mean square's error halves in the root, then the division, the sum with eps,
# root and reciprocal: rstd is off by less than this, relatively.
D_R = (ADDS + 2) / 2 * U + 4 * U

SIZES = [(1, 1), (1, 7), (3, 8), (5, 64), (33, 72), (7, 128), (9, 136), (2, 255), (9, 256), (130, 264), (17, 512),
         (33, 513), (5, 1023), (300, 1024), (2, 1600), (700, 2048), (3, 4095), (64, 4096), (2, 4104), (400, 5000),
         (5, 8192), (3, 8200), (2, 16384), (2, 16385), (3, 32768), (2, 40000)]


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


def draw(rows, dim, xt, wt, seed):
    gen = torch.Generator().manual_seed(seed)
    x, r, dy, dh = ((torch.randn((rows, dim), generator=gen) * s).to(xt) for s in (2.0, 1.0, 1.0, 1.0))
    w = (1 + 0.3 * torch.randn(dim, generator=gen)).to(wt)
    return [t.to(DEV) for t in (x, r, dy, dh, w)]


def moved(t):
    """The same values one element off the 16-byte grid."""
    flat = torch.empty(t.numel() + 1, dtype=t.dtype, device=DEV)
    flat[1:].copy_(t.reshape(-1))
    return flat[1:].reshape(t.shape)


def stream64(x, r):
    """H: the sum rounded to the type (fp32's own addition for 16-bit types is exact to 2^-24 of it)."""
    return x if r is None else (x.float() + r.float()).to(x.dtype)


def check_forward(g, x, w, r):
    Y, H, rstd = g.rms_norm_fwd(x, w, residual=r, eps=EPS)
    Y2, H2, none = g.rms_norm_fwd(x, w, residual=r, eps=EPS, stats=False)
    assert g.check() == g.GEMM_OK and none is None
    assert torch.equal(Y, Y2) and torch.equal(H, H2) and torch.equal(H, stream64(x, r))
    h = H.double()
    want_r = 1 / torch.sqrt((h * h).mean(-1) + EPS)
    assert ((rstd.double() - want_r).abs() <= D_R * want_r).all()
    y = h * want_r[..., None] * (1.0 if w is None else w.double())
    rel, tiny = half_step(x.dtype)
    assert ((Y.double() - y).abs() <= (D_R + 3 * U + rel) * 1.001 * y.abs() + tiny).all()
    return H, rstd, y


def check_fp8(g, x, w, r, pow2):
    Q, S, H = g.rms_norm_fp8(x, w, residual=r, eps=EPS, pow2=pow2)
    assert g.check() == g.GEMM_OK and torch.equal(H, stream64(x, r))
    h = H.double()
    y = h / torch.sqrt((h * h).mean(-1, keepdim=True) + EPS) * (1.0 if w is None else w.double())
    rows, dim = x.shape
    a = ref.blocks(y, 1).abs().amax(dim=(1, 3))
    d = D_R + 3 * U   # of y, and so of a
    if pow2:
        s = torch.exp2(S.double() - 127)
        assert ((a * (1 - d) <= 448 * s) & ((a * (1 + d) > 224 * s) | (a == 0))).all()
    else:
        s = S.double()
        want = torch.where(a > 0, a / 448, torch.ones_like(a))
        assert ((s - want).abs() <= (d + U) * 1.001 * want + 2.0 ** -149).all()
    # y / s as the kernel has it: y's error, the quotient's rounding, and with fp32
    # scales the scale's own.
    v = y / ref.spread(s, 1, rows, dim)
    err = (2 * d + 4 * U) * 1.001 * v.abs()
    got = Q.float().double()
    assert ((got - v).abs() <= ref.e4m3_half_step(v.abs() + err) + err).all()
    assert (got.abs() <= 448).all()


def check_backward(g, x, dy, w, rstd, wt, dh):
    dX, dg = g.rms_norm_bwd(dy, x, rstd, w, dH=dh, wtype=wt if w is None else None)
    dX2, none = g.rms_norm_bwd(dy, x, rstd, w, dH=dh, weights=False)
    assert g.check() == g.GEMM_OK and none is None and torch.equal(dX, dX2) and dg.dtype == wt
    r, d = rstd.double()[:, None], dy.double()
    z = x.double() * r
    gr = d if w is None else d * w.double()
    c = (gr * z).mean(-1, keepdim=True)
    base = 0.0 if dh is None else dh.double()
    want = base + r * (gr - z * c)
    d_c = (ADDS + 5) * U * (gr * z).abs().mean(-1, keepdim=True)
    rel, tiny = half_step(x.dtype)
    tol = r * (z.abs() * d_c + 6 * U * (gr.abs() + (z * c).abs())) + 2 * U * want.abs()
    assert ((dX.double() - want).abs() <= 1.01 * (tol + rel * want.abs() + tiny)).all()
    rel, tiny = half_step(wt)
    terms = d * z
    s = terms.sum(0)
    # rows of a block one by one, then the blocks' sums
    tol = (ADDS + 3) * U * terms.abs().sum(0) + rel * s.abs() + tiny
    assert ((dg.double() - s).abs() <= 1.01 * tol).all()
    return dX, dg


@pytest.mark.parametrize("xt,wt", TYPES)
@pytest.mark.parametrize("rows,dim", SIZES)
def test_forward_and_backward(g, rows, dim, xt, wt):
    x, r, dy, dh, w = draw(rows, dim, DTYPES[xt], DTYPES[wt], rows * 31 + dim)
    check_forward(g, x, w, None)
    H, rstd, _ = check_forward(g, x, w, r)
    check_backward(g, H, dy, w, rstd, DTYPES[wt], dh)
    check_backward(g, H, dy, w, rstd, DTYPES[wt], None)


@pytest.mark.parametrize("pow2", [False, True])
@pytest.mark.parametrize("xt,wt", TYPES)
@pytest.mark.parametrize("rows,dim", SIZES)
def test_fp8_output(g, rows, dim, xt, wt, pow2):
    x, r, _, _, w = draw(rows, dim, DTYPES[xt], DTYPES[wt], rows * 37 + dim)
    check_fp8(g, x, w, r, pow2)
    check_fp8(g, x, w, None, pow2)


@pytest.mark.parametrize("xt,wt", TYPES)
@pytest.mark.parametrize("dim", [96, 1000, 2056])
def test_without_weights(g, dim, xt, wt):
    x, r, dy, dh, w = draw(21, dim, DTYPES[xt], DTYPES[wt], dim)
    H, rstd, _ = check_forward(g, x, None, r)
    check_backward(g, H, dy, None, rstd, DTYPES[wt], dh)
    check_fp8(g, x, None, r, False)


@pytest.mark.parametrize("xt,wt", TYPES)
@pytest.mark.parametrize("dim", [64, 2048, 2050])
def test_unaligned_buffers(g, dim, xt, wt):
    x, r, dy, dh, w = (moved(t) for t in draw(10, dim, DTYPES[xt], DTYPES[wt], 3))
    H, rstd, _ = check_forward(g, x, w, r)
    check_backward(g, moved(H), dy, w, rstd, DTYPES[wt], dh)
    check_fp8(g, x, w, r, False)
    # an output off the grid beside aligned inputs
    x, r, dy, dh, w = draw(10, dim, DTYPES[xt], DTYPES[wt], 3)
    Q = torch.empty(10 * dim + 1, dtype=torch.uint8, device=DEV)[1:].view(torch.float8_e4m3fn).reshape(10, dim)
    want = g.rms_norm_fp8(x, w, residual=r, eps=EPS)
    got = g.rms_norm_fp8(x, w, residual=r, eps=EPS, Q=Q)
    assert ref.e4m3_half_step(got[0].double()).shape == (10, dim)
    # another division of the row's sum among threads: rstd may differ by its tolerance
    same = (got[0].view(torch.uint8) == want[0].view(torch.uint8)).double().mean()
    assert same > 0.99 and torch.equal(got[2], want[2])


@pytest.mark.parametrize("rows,dim", [(5000, 128), (4097, 1030), (3000, 40), (2500, 1024), (2000, 4096), (900, 5000)])
def test_more_rows_than_blocks(g, rows, dim):
    x, r, dy, dh, w = draw(rows, dim, torch.float16, torch.float32, 7)
    H, rstd, _ = check_forward(g, x, w, r)
    r64, d = rstd.double()[:, None], dy.double()
    dX, dg = g.rms_norm_bwd(dy, H, rstd, w, dH=dh)
    assert g.check() == g.GEMM_OK
    terms = d * H.double() * r64
    # a block has at most rows / 152 + 1 of them one by one
    tol = (rows / 152 + 20) * U * terms.abs().sum(0) + U * terms.sum(0).abs()
    assert ((dg.double() - terms.sum(0)).abs() <= 1.01 * tol).all()
    c = (terms * w.double()).mean(-1, keepdim=True)
    want = dh.double() + r64 * (d * w.double() - H.double() * r64 * c)
    assert ((dX.double() - want).abs() <= 2.0 ** -10 * (want.abs() + 2.0 ** -6)).all()


@pytest.mark.parametrize("xt", list(DTYPES))
@pytest.mark.parametrize("dim", [100, 4096, 4097, 40000])
def test_stream_updated_in_place(g, dim, xt):
    x, r, _, _, w = draw(9, dim, DTYPES[xt], DTYPES[xt], dim)
    Y, H, rstd = g.rms_norm_fwd(x, w, residual=r, eps=EPS)
    Q, S, _ = g.rms_norm_fp8(x, w, residual=r, eps=EPS)
    for which in (0, 1):
        pair = [x.clone(), r.clone()]
        y, h, s = g.rms_norm_fwd(pair[0], w, residual=pair[1], eps=EPS, H=pair[which])
        assert h is pair[which] and torch.equal(h, H) and torch.equal(y, Y) and torch.equal(s, rstd)
        pair = [x.clone(), r.clone()]
        q, s, h = g.rms_norm_fp8(pair[0], w, residual=pair[1], eps=EPS, H=pair[which])
        assert torch.equal(q.view(torch.uint8), Q.view(torch.uint8)) and torch.equal(s, S) and torch.equal(h, H)
        assert torch.equal(pair[1 - which], r if which == 0 else x)
    both = x.clone()
    _, h, _ = g.rms_norm_fwd(both, w, residual=both, eps=EPS, H=both)
    assert torch.equal(h, (x.float() * 2).to(x.dtype))
    assert g.check() == g.GEMM_OK


def test_zero_rows_and_large_and_small_values(g):
    x = torch.zeros((4, 512), device=DEV, dtype=torch.bfloat16)
    x[1] = 1e-18
    x[2] = 3e18
    x[3, 7] = 2.0
    Y, _, rstd = g.rms_norm_fwd(x, eps=EPS)
    assert (Y[0] == 0).all() and torch.isfinite(Y).all() and abs(float(Y[2, 0]) - 1) < 2 ** -7
    Q, S, _ = g.rms_norm_fp8(x, eps=EPS)
    assert (Q[0].float() == 0).all() and (S[0] == 1).all()
    assert (S[3, 1:] == 1).all() and float(Q[3, 7].float()) == 448.0
    Q, S, _ = g.rms_norm_fp8(x, eps=EPS, pow2=True)
    assert (S[0] == 127).all() and (S[3, 1:] == 127).all()
    assert g.check() == g.GEMM_OK


@pytest.mark.parametrize("dim", [96, 1000, 1001, 20001])
def test_infinities_and_nan_are_not_hidden(g, dim):
    x = torch.randn((3, dim), device=DEV).half()
    x[0, dim - 1] = float("nan")
    x[1, 0] = float("inf")
    Q, S, _ = g.rms_norm_fp8(x, eps=EPS)
    # NaN everywhere in the row: its mean square is
    assert torch.isnan(S[0]).all() and torch.isnan(Q[0].float()).all()
    # inf * 0 in its own place, 0 elsewhere
    assert torch.isnan(S[1, 0]) and torch.isnan(Q[1, :min(dim, 128)].float()).all()
    assert torch.isfinite(S[2]).all() and torch.isfinite(Q[2].float()).all()
    _, S, _ = g.rms_norm_fp8(x, eps=EPS, pow2=True)
    assert (S[0] == 255).all() and S[1, 0] == 255 and (S[2] != 255).all()


def test_leading_dimensions_and_empty(g):
    x = torch.randn((2, 3, 5, 96), device=DEV).half()
    Y, H, rstd = g.rms_norm_fwd(x, residual=x)
    assert Y.shape == x.shape and rstd.shape == x.shape[:-1]
    y, h, r = g.rms_norm_fwd(x.reshape(-1, 96), residual=x.reshape(-1, 96))
    assert torch.equal(y.reshape(x.shape), Y) and torch.equal(r.reshape(rstd.shape), rstd)
    Q, S, _ = g.rms_norm_fp8(x)
    assert Q.shape == x.shape and S.shape == (2, 3, 5, 1)
    e = torch.empty((0, 96), device=DEV).half()
    Y, H, rstd = g.rms_norm_fwd(e)
    assert Y.shape == e.shape and rstd.shape == (0,)
    w = torch.ones(96, device=DEV).half()
    dX, dg = g.rms_norm_bwd(e, e, rstd, w)
    assert dX.shape == e.shape and (dg == 0).all()
    e = torch.empty((4, 0), device=DEV).half()
    assert g.rms_norm_fwd(e)[0].shape == (4, 0) and g.rms_norm_fp8(e)[1].shape == (4, 0)


def test_refusals(g):
    x = torch.randn((8, 64), device=DEV).half()
    r = torch.randn((8, 64), device=DEV).half()
    buf = torch.empty(8 * 64 + 64, device=DEV).half()
    with pytest.raises(g.GemmError):   # half a row further than X
        g.rms_norm_fwd(buf[:512].reshape(8, 64), residual=r, H=buf[32:544].reshape(8, 64))
    with pytest.raises(g.GemmError):
        g.rms_norm_fwd(x, residual=r, Y=x)
    with pytest.raises(g.GemmError):
        g.rms_norm_fwd(x, residual=r, H=r, Y=r)
    Y, H, rstd = g.rms_norm_fwd(x, residual=r)
    with pytest.raises(g.GemmError):
        g.rms_norm_bwd(x, H, rstd, dX=H)
    with pytest.raises(g.GemmError):
        g.rms_norm_bwd(x, H, rstd, workspace=torch.empty(4, device=DEV))
    with pytest.raises(ValueError):
        g.rms_norm_fwd(x, residual=r.cpu())
    with pytest.raises(g.GemmError):
        g.rms_norm_fwd(x, eps=-1.0)
    assert g.check() == g.GEMM_OK


@pytest.mark.parametrize("xt,rows,dim", [("fp16", 3, 1024), ("fp16", 700, 4096), ("bf16", 400, 5000),
                                         ("fp16", 40, 16384), ("fp32", 400, 2047), ("fp16", 400, 4100), ("fp32", 7, 8192)])
def test_wait_runs_out_and_context_survives(g, xt, rows, dim):
    x, r, dy, dh, w = draw(rows, dim, DTYPES[xt], DTYPES[xt], dim)
    H, rstd, _ = check_forward(g, x, w, r)
    dX = torch.full_like(x, 5.0)
    assert g.check() == g.GEMM_OK
    st = g.lib().rms_norm_bwd_selftest_timeout(dy.data_ptr(), H.data_ptr(), rstd.data_ptr(), dX.data_ptr(), rows, dim,
                                               g.TYPES[x.dtype], 1 << 20, torch.cuda.current_stream().cuda_stream)
    assert st == g.GEMM_OK
    assert g.check() == g.GEMM_ERR_TIMEOUT
    assert (g.last_timeout_record() & 0xFF) == 9, hex(g.last_timeout_record())
    assert (dX == 5.0).all()
    check_backward(g, H, dy, w, rstd, w.dtype, dh)


@pytest.mark.parametrize("dim", [24, 96, 1056])
def test_gradients_against_differences(g, dim):
    """A sum of outputs and stream, weighted, moved along random directions, in fp32."""
    gen = torch.Generator().manual_seed(dim)
    x, r, cy, ch, vx, vr = (torch.randn((4, dim), generator=gen).to(DEV) for _ in range(6))
    w, vw = (torch.randn(dim, generator=gen).to(DEV) for _ in range(2))

    def value(t):
        # in 64 bits: the kernel's own values would differ by their rounding over the step
        h = (x + r).double() + t * (vx + vr).double()
        y = h / torch.sqrt((h * h).mean(-1, keepdim=True) + EPS) * (w.double() + t * vw.double())
        return ((y * cy.double()).sum() + (h * ch.double()).sum()).item()

    t = 1e-5
    slope = (value(t) - value(-t)) / (2 * t)
    _, H, rstd = g.rms_norm_fwd(x, w, residual=r, eps=EPS)
    dX, dg = g.rms_norm_bwd(cy, H, rstd, w, dH=ch)
    got = ((dX.double() * (vx + vr).double()).sum() + (dg.double() * vw.double()).sum()).item()
    # The difference's own error, about t^2 of the third derivative, and 4 dim terms
    # of size about one with fp32's rounding.
    assert abs(got - slope) <= 1e-4 * (1 + abs(slope)) + 4 * dim * (ADDS + 8) * U


@pytest.mark.parametrize("xt", ["bf16", "fp32"])
@pytest.mark.parametrize("dim", [40, 100, 512, 1001, 4096, 20001])
def test_rows_whose_squares_are_beyond_fp32(g, dim, xt):
    gen = torch.Generator().manual_seed(dim)
    scale = torch.tensor([1.0, 1e19, 1e30, 1e37, 1e-30]).reshape(5, 1)
    x = (torch.randn((5, dim), generator=gen).clamp(-4, 4) * scale).to(DTYPES[xt]).to(DEV)
    Y, _, rstd = g.rms_norm_fwd(x, eps=EPS)
    Q, S, _ = g.rms_norm_fp8(x, eps=EPS)
    assert g.check() == g.GEMM_OK
    h = x.double()
    r = 1 / torch.sqrt((h * h).mean(-1) + EPS)
    # rstd below 2^-126 has steps of 2^-149
    assert ((rstd.double() - r).abs() <= D_R * r + 2.0 ** -149).all()
    y = h * r[:, None]
    rel, tiny = half_step(x.dtype)
    d = D_R + 2.0 ** -149 / r + 3 * U
    assert ((Y.double() - y).abs() <= (d[:, None] + rel) * 1.001 * y.abs() + tiny).all()
    v = Q.float().double() * ref.spread(S.double(), 1, 5, dim)
    a = ref.spread(ref.blocks(y, 1).abs().amax(dim=(1, 3)), 1, 5, dim)
    assert ((v - y).abs() <= 2.0 ** -4 * 1.001 * y.abs() + a * 2.0 ** -17).all()


def check_many_rows(g, H, dy, w, rstd, dh, dX=None):
    """Gradients of more rows than a block has: a block adds at most rows / 152 + 8 of them one by one."""
    rows = H.shape[0]
    r, d = rstd.double()[:, None], dy.double()
    z = H.double() * r
    dX, dg = g.rms_norm_bwd(dy, H, rstd, w, dH=dh, dX=dX)
    assert g.check() == g.GEMM_OK
    terms = d * z
    rel, tiny = half_step(w.dtype)
    tol = (rows / 152 + 24) * U * terms.abs().sum(0) + rel * terms.sum(0).abs() + tiny
    assert ((dg.double() - terms.sum(0)).abs() <= 1.01 * tol).all()
    gr = d * w.double()
    c = (gr * z).mean(-1, keepdim=True)
    want = r * (gr - z * c) + (0.0 if dh is None else dh.double())
    rel, tiny = half_step(H.dtype)
    d_c = (ADDS + 5) * U * (gr * z).abs().mean(-1, keepdim=True)
    tol = r * (z.abs() * d_c + 6 * U * (gr.abs() + (z * c).abs())) + 2 * U * want.abs()
    assert ((dX.double() - want).abs() <= 1.01 * (tol + rel * want.abs() + tiny)).all()
    return dX, dg


@pytest.mark.parametrize("xt,wt,rows,dim", [
    ("fp16", "fp16", 400, 16384), ("fp32", "fp32", 400, 16384), ("bf16", "fp32", 700, 12000), ("fp32", "fp32", 333, 16377),
    ("bf16", "bf16", 500, 16370), ("bf16", "bf16", 200, 16371), ("fp16", "fp32", 700, 9001), ("fp16", "fp16", 1300, 4097),
    ("bf16", "fp32", 1300, 4999), ("fp32", "fp32", 900, 3001), ("bf16", "bf16", 4000, 1023), ("fp32", "fp32", 2000, 513),
    ("fp16", "fp16", 2001, 514), ("fp32", "fp32", 305, 2), ("fp16", "fp16", 153, 1025), ("fp16", "fp16", 305, 1025)])
def test_rows_of_any_width_more_than_blocks(g, xt, wt, rows, dim):
    x, _, dy, dh, w = draw(rows, dim, DTYPES[xt], DTYPES[wt], rows + dim)
    _, H, rstd = g.rms_norm_fwd(x, w, eps=EPS)
    first = check_many_rows(g, H, dy, w, rstd, dh)
    check_many_rows(g, H, dy, w, rstd, None)
    # all four off the 16-byte grid by the same element, then by different ones
    off = torch.empty(rows * dim + 1, dtype=x.dtype, device=DEV)[1:].reshape(rows, dim)
    same = check_many_rows(g, moved(H), moved(dy), moved(w), rstd, moved(dh), dX=off)
    other = check_many_rows(g, moved(H), dy, w, rstd, dh, dX=off.clone())
    for got in (same, other):   # the same sums, divided among threads another way
        assert got[0].shape == first[0].shape and got[1].dtype == first[1].dtype


@pytest.mark.parametrize("xt,dim", [("fp16", 1025), ("bf16", 4099), ("fp32", 2047), ("fp16", 16369)])
def test_nothing_beside_the_rows_is_read_or_written(g, xt, dim):
    """NaN in front of the first and behind the last row, and in the 16-byte pieces that they share."""
    rows = 7
    x, _, dy, dh, w = draw(rows, dim, DTYPES[xt], DTYPES[xt], dim)
    _, H, rstd = g.rms_norm_fwd(x, w, eps=EPS)
    want = g.rms_norm_bwd(dy, H, rstd, w, dH=dh)

    def inside(t, by):
        flat = torch.full((t.numel() + 64,), float("nan"), dtype=t.dtype, device=DEV)
        part = flat[by:by + t.numel()].reshape(t.shape)
        part.copy_(t)
        return flat, part

    for by in (0, 1, 3, 8):
        flat, out = inside(torch.zeros_like(H), by)
        got = g.rms_norm_bwd(inside(dy, by)[1], inside(H, by)[1], rstd, w, dH=inside(dh, by)[1], dX=out)
        assert g.check() == g.GEMM_OK
        assert torch.isfinite(got[0]).all() and torch.isfinite(got[1]).all()
        assert torch.isnan(flat[:by]).all() and torch.isnan(flat[by + H.numel():]).all()
        rel, tiny = half_step(H.dtype)
        # another division of the row's sum among threads may turn a rounding
        assert ((got[0].double() - want[0].double()).abs()
                <= 2 * rel * want[0].double().abs() + 2.0 ** -18 * want[0].double().abs().max()).all()


@pytest.mark.parametrize("xt,wt,rows,dim", [
    ("fp16", "fp16", 1300, 4097), ("bf16", "fp32", 1300, 4098), ("bf16", "bf16", 300, 16371), ("bf16", "bf16", 300, 16369),
    ("fp16", "fp32", 5600, 769), ("fp32", "fp32", 2100, 4095), ("fp32", "fp32", 1000, 8389), ("fp16", "fp16", 2100, 2048),
    ("fp16", "fp16", 2098, 2047)])
def test_many_rows_of_any_width_forward(g, xt, wt, rows, dim):
    x, r, _, _, w = draw(rows, dim, DTYPES[xt], DTYPES[wt], rows + dim)
    check_forward(g, x, w, None)
    check_forward(g, x, None, r)
    want = g.rms_norm_fwd(x, w, residual=r, eps=EPS)
    total = rows * dim

    def beside(t, by):
        """t's values among NaNs, `by` elements off the 16-byte grid."""
        flat = torch.full((total + 64,), float("nan"), dtype=t.dtype, device=DEV)
        flat[by:by + total].copy_(t.reshape(-1))
        return flat, flat[by:by + total].reshape(rows, dim)

    check_forward(g, moved(x), moved(w), moved(r))
    for by in (0, 3):
        for which in (0, 1):   # the stream in the place of either summand
            fx, px = beside(x, by)
            fr, pr = beside(r, by)
            fy, py = beside(torch.zeros_like(x), by)
            Y, H, _ = g.rms_norm_fwd(px, w, residual=pr, eps=EPS, Y=py, H=(px, pr)[which])
            assert g.check() == g.GEMM_OK
            rel, tiny = half_step(x.dtype)
            # another division of the row's sum among threads may turn a rounding
            step = (2 * rel + 2 * D_R) * want[0].double().abs() + tiny
            assert torch.equal(H, want[1]) and ((Y.double() - want[0].double()).abs() <= step).all()
            for flat in (fx, fr, fy):
                assert torch.isnan(flat[:by]).all() and torch.isnan(flat[by + total:]).all()
            assert torch.equal((pr, px)[which], (r, x)[which])


@pytest.mark.parametrize("dim", [4097, 8191])
def test_many_rows_beyond_fp32_squares(g, dim):
    gen = torch.Generator().manual_seed(dim)
    scale = torch.tensor([1.0, 1e19, 1e30, 1e-30, 1.0]).repeat(260).reshape(-1, 1)
    x = (torch.randn((1300, dim), generator=gen).clamp(-4, 4) * scale).to(torch.bfloat16).to(DEV)
    x[4, 7], x[9, dim - 1] = float("inf"), float("nan")
    Y, _, rstd = g.rms_norm_fwd(x, eps=EPS)
    assert g.check() == g.GEMM_OK
    good = torch.ones(1300, dtype=torch.bool, device=DEV)
    good[4] = good[9] = False
    h = x[good].double()
    want_r = 1 / torch.sqrt((h * h).mean(-1) + EPS)
    assert ((rstd[good].double() - want_r).abs() <= D_R * want_r + 2.0 ** -149).all()
    assert rstd[4] == 0 and torch.isnan(rstd[9])
    assert torch.isnan(Y[4, 7]) and (Y[4, 8:] == 0).all() and torch.isnan(Y[9]).all()
