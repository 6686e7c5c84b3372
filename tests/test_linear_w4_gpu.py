"""GPU tests of 4-bit weights with group scales: quantisation, layout and product
against the definitions in 64 bits."""
from __future__ import annotations

import pytest
import torch

import feed_forward_reference as ref

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda:0")
DTYPES = {"fp16": torch.float16, "bf16": torch.bfloat16, "fp32": torch.float32}
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


def packed(g, N, K, group, zeros, dtype, seed):
    gen = torch.Generator().manual_seed(seed)
    q = torch.randint(0, 16, (N, K), generator=gen, dtype=torch.uint8)
    s = (torch.exp(0.5 * torch.randn((N, -(-K // group)), generator=gen)) / K ** 0.5).to(dtype)
    z = torch.randint(0, 16, s.shape, generator=gen, dtype=torch.uint8) if zeros else None
    return g.w4_pack(q.to(DEV), s.to(DEV), None if z is None else z.to(DEV), group)


def check(g, X, W, N, group, relu):
    C = g.linear_w4(X, *W, N=N, group=group, relu=relu)
    assert g.check() == g.GEMM_OK and C.shape == (X.shape[0], N) and C.dtype == X.dtype
    K = X.shape[1]
    w = ref.weight_w4(*W, N, K, group)
    x = X.double()
    y = x @ w.t()
    want = y.clamp(min=0) if relu else y
    # q - z is exact and so is its product with x.  A product of 16 columns may cut
    # each of its 17 summands to a step of 2^-23 of the largest; eight of them make
    # up a group, then the groups' and the warps' and blocks' sums are rounded.
    steps = 2 * 17 * 8 + 2 * (K // 128 + 1) + 80
    tol = steps * U * (x.abs() @ w.abs().t()) + torch.finfo(X.dtype).eps / 2 * want.abs() + 2.0 ** -25
    assert ((C.double() - want).abs() <= 1.01 * tol).all()
    assert torch.equal(C, g.linear_w4(X, *W, N=N, group=group, relu=relu))
    return C


SIZES = [(1, 1, 1), (1, 16, 64), (1, 17, 65), (2, 64, 128), (3, 100, 129), (7, 48, 200), (8, 256, 1024), (9, 33, 1000),
         (1, 4096, 4096), (16, 130, 2056), (17, 64, 4097), (31, 500, 320), (33, 80, 640), (64, 264, 1032), (1, 40, 16384),
         (5, 2000, 999), (64, 16, 8192), (4, 3000, 4104)]


@pytest.mark.parametrize("xt", ["fp16", "bf16"])
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("zeros", [False, True])
@pytest.mark.parametrize("M,N,K", SIZES)
def test_product(g, M, N, K, group, zeros, xt):
    W = packed(g, N, K, group, zeros, DTYPES[xt], M + N + K)
    gen = torch.Generator().manual_seed(K)
    X = torch.randn((M, K), generator=gen).to(DTYPES[xt]).to(DEV)
    check(g, X, W, N, group, relu=(M + N) % 2 == 0)


@pytest.mark.parametrize("xt", ["fp16", "bf16"])
def test_every_code_and_zero_point(g, xt):
    """Each code with each zero point in every place of a tile, scales of one: the sum is exact."""
    K = 128
    for z in range(16):
        q = ((torch.arange(32)[:, None] * 5 + torch.arange(K)[None, :] * 3) % 16).to(torch.uint8).to(DEV)
        s = torch.ones((32, 2), dtype=DTYPES[xt], device=DEV)
        W = g.w4_pack(q, s, torch.full((32, 2), z, dtype=torch.uint8, device=DEV), 64)
        for k in range(0, K, 9):
            X = torch.zeros((2, K), dtype=DTYPES[xt], device=DEV)
            X[1, k] = 1.0
            C = g.linear_w4(X, *W, group=64)
            assert (C[0] == 0).all() and torch.equal(C[1].double(), q[:, k].double() - z)
    assert g.check() == g.GEMM_OK


def test_pack_is_the_documented_layout(g):
    gen = torch.Generator().manual_seed(2)
    q = torch.randint(0, 16, (37, 200), generator=gen, dtype=torch.uint8).to(DEV)
    s = torch.randn((37, 7), generator=gen).half().to(DEV)
    Q, S, Z = g.w4_pack(q, s, None, 32)
    assert Z is None and Q.shape == (3, 4, 512) and S.shape == (3, 7, 16)
    assert torch.equal(ref.unpack_w4(Q, 37, 200), q.long())
    assert torch.equal(ref.per_column(S, 37, 200, 32)[:, ::32], s.double())


@pytest.mark.parametrize("wt", list(DTYPES))
@pytest.mark.parametrize("st", ["fp16", "bf16"])
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("N,K,transpose", [(1, 1, False), (40, 200, False), (17, 129, True), (128, 512, True)])
def test_quantisation(g, N, K, transpose, group, st, wt):
    gen = torch.Generator().manual_seed(N + K)
    w = torch.randn((N, K), generator=gen)
    w[0, :group] = 0.0
    w = (w * torch.exp(torch.randn((N, 1), generator=gen))).to(DTYPES[wt]).to(DEV)
    stored = w.t().contiguous() if transpose else w
    rel = torch.finfo(DTYPES[st]).eps / 2
    groups = -(-K // group)
    full = torch.zeros((N, groups * group), dtype=torch.float64, device=DEV)
    full[:, :K] = w.double()
    per = full.reshape(N, groups, group)
    for zeros in (False, True):
        Q, S, Z = g.w4_quantize(stored, group, zeros, transpose, DTYPES[st])
        assert g.check() == g.GEMM_OK
        s = ref.per_column(S, N, groups * group, group)[:, ::group]
        lo, hi = per.amin(2).clamp(max=0), per.amax(2).clamp(min=0)
        want = (hi - lo) / 15 if zeros else per.abs().amax(2) / 7
        # rounded to the scales' type after at most four roundings in fp32
        assert ((s - want).abs() <= (rel + 4 * U) * want + 2.0 ** -25).all()
        sk = ref.per_column(S, N, K, group)
        if zeros:
            z = ref.per_column(Z, N, groups * group, group)[:, ::group]
            v = torch.where(s > 0, -lo / s, torch.zeros_like(s))
            assert ((z - v.clamp(0, 15)).abs() <= 0.5 + 8 * U * 16).all()
            zk = ref.per_column(Z, N, K, group)
        else:
            assert Z is None
            zk = 8.0
        q = ref.unpack_w4(Q, N, K).double()
        v = torch.where(sk > 0, w.double() / sk, torch.zeros_like(sk))
        # w / s to the nearest whole number, then kept in 0 .. 15
        assert ((q - (v + zk).clamp(0, 15)).abs() <= 0.5 + 2 * U * 16).all()
        # What fills up the tiles is zero.
        full_q = ref.unpack_w4(Q, Q.shape[0] * 16, Q.shape[1] * 64)
        assert (full_q[N:] == 0).all() and (full_q[:, K:] == 0).all()


def test_quantisation_of_infinities_nan_and_extremes(g):
    w = torch.randn((16, 256), device=DEV)
    w[0, 3], w[1, 200], w[2, :128] = float("nan"), float("inf"), 1e30
    w[3, :128] = 1e-30
    Q, S, Z = g.w4_quantize(w, 128)
    s = ref.per_column(S, 16, 256, 128)[:, ::128]
    assert torch.isnan(s[0, 0]) and torch.isnan(s[1, 1]) and int(torch.isnan(s).sum()) == 2
    assert s[2, 0] == 65504.0 and s[3, 0] == 0.0
    q = ref.unpack_w4(Q, 16, 256)
    assert (q[2, :128] == 15).all() and (q[3, :128] == 8).all()
    X = torch.ones((1, 256), device=DEV).half()
    C = g.linear_w4(X, Q, S)
    assert torch.isnan(C[0, :2]).all() and torch.isfinite(C[0, 3:]).all()


def test_rows_of_x_do_not_reach_one_another(g):
    """A row with an infinity or a NaN leaves the others' results as they are."""
    W = packed(g, 96, 512, 64, True, torch.float16, 1)
    X = torch.randn((24, 512), device=DEV).half()
    want = g.linear_w4(X, *W, group=64)
    X[5, 100], X[17, 0] = float("inf"), float("nan")
    got = g.linear_w4(X, *W, group=64)
    rows = [i for i in range(24) if i not in (5, 17)]
    assert torch.equal(got[rows], want[rows])
    assert not torch.isfinite(got[5]).any() and torch.isnan(got[17]).all()


def test_unaligned_activations(g):
    for t in (torch.float16, torch.bfloat16):
        W = packed(g, 80, 512, 128, False, t, 4)
        X = torch.randn((6, 512), device=DEV).to(t)
        flat = torch.empty(6 * 512 + 1, dtype=t, device=DEV)
        flat[1:].copy_(X.reshape(-1))
        assert torch.equal(g.linear_w4(flat[1:].reshape(6, 512), *W), g.linear_w4(X, *W))


def test_rows_past_the_output_are_left_alone(g):
    W = packed(g, 50, 256, 64, False, torch.float16, 4)
    X = torch.randn((3, 256), device=DEV).half()
    buf = torch.full((5 * 50,), 7.0, device=DEV).half()
    C = buf[50:200].reshape(3, 50)
    assert torch.equal(g.linear_w4(X, *W, N=50, group=64, C=C), g.linear_w4(X, *W, N=50, group=64))
    assert (buf[:50] == 7).all() and (buf[200:] == 7).all()


def test_empty_and_refused(g):
    W = packed(g, 32, 128, 64, False, torch.float16, 4)
    X = torch.zeros((2, 128), device=DEV).half()
    assert g.linear_w4(X[:0], *W, group=64).shape == (0, 32)
    none = g.w4_pack(torch.zeros((32, 0), dtype=torch.uint8, device=DEV), torch.zeros((32, 0), device=DEV).half())
    assert (g.linear_w4(torch.zeros((2, 0), device=DEV).half(), *none) == 0).all()
    with pytest.raises(ValueError):
        g.linear_w4(torch.zeros((65, 128), device=DEV).half(), *W, group=64)
    with pytest.raises(ValueError):   # scales of another type
        g.linear_w4(X.bfloat16(), *W, group=64)
    with pytest.raises(ValueError):   # the packed form of another group or K
        g.linear_w4(X, *W, group=128)
    with pytest.raises(ValueError):
        g.linear_w4(torch.zeros((2, 192), device=DEV).half(), *W, group=64)
    with pytest.raises(ValueError):
        g.linear_w4(X, *W, group=48)
    with pytest.raises(ValueError):
        g.linear_w4(X, *W, N=50, group=64)
    with pytest.raises(g.GemmError):
        g.linear_w4(X, *W, group=64, C=X.reshape(-1)[:64].reshape(2, 32))
    assert g.check() == g.GEMM_OK


# More than 32 rows of X go to the tensor memory kernel: blocks of 128 rows of W, walked
# by the GPU's 152 blocks or one to a block or a cluster; units of 128 columns.
MANY = [(33, 1, 1), (33, 20000, 100), (64, 19600, 130), (40, 128, 128), (50, 129, 300), (48, 1000, 2184), (64, 2048, 6000),
        (37, 260, 8191), (64, 4100, 1024), (64, 9728, 520), (35, 38912, 64), (63, 640, 16384)]


@pytest.mark.parametrize("xt", ["fp16", "bf16"])
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("zeros", [False, True])
@pytest.mark.parametrize("M,N,K", MANY)
def test_many_rows_of_activations(g, M, N, K, group, zeros, xt):
    W = packed(g, N, K, group, zeros, DTYPES[xt], M + N + K)
    gen = torch.Generator().manual_seed(K)
    X = torch.randn((M, K), generator=gen).to(DTYPES[xt]).to(DEV)
    C = check(g, X, W, N, group, relu=(M + N) % 2 == 0)
    # off the 16-byte grid, between other tensors' bytes: the same products and sums
    flat = torch.full((M * K + 2,), float("nan"), dtype=X.dtype, device=DEV)
    flat[1:-1].copy_(X.reshape(-1))
    buf = torch.full((M * N + 64,), 7.0, dtype=X.dtype, device=DEV)
    out = buf[32:32 + M * N].reshape(M, N)
    assert torch.equal(g.linear_w4(flat[1:-1].reshape(M, K), *W, N=N, group=group, relu=(M + N) % 2 == 0, C=out), C)
    assert (buf[:32] == 7).all() and (buf[32 + M * N:] == 7).all()


@pytest.mark.parametrize("M", [33, 64])
def test_columns_reach_their_own_products(g, M):
    """One activation at a time: every column of W, in its own place, with its own sign and group."""
    K, N, group = 256, 144, 64
    gen = torch.Generator().manual_seed(M)
    q = torch.randint(0, 16, (N, K), generator=gen, dtype=torch.uint8)
    s = torch.exp2(torch.randint(-3, 4, (N, K // group), generator=gen).float()).half()
    z = torch.randint(0, 16, s.shape, generator=gen, dtype=torch.uint8)
    W = g.w4_pack(q.to(DEV), s.to(DEV), z.to(DEV), group)
    w = (q.double() - z.double().repeat_interleave(group, 1)) * s.double().repeat_interleave(group, 1)
    for k0 in range(0, K, M):
        n = min(M, K - k0)
        X = torch.zeros((M, K), dtype=torch.float16)
        X[torch.arange(n), k0 + torch.arange(n)] = 1.0
        C = g.linear_w4(X.to(DEV), *W, N=N, group=group)
        assert torch.equal(C[:n].double().cpu(), w[:, k0:k0 + n].t()) and (C[n:] == 0).all()
    assert g.check() == g.GEMM_OK


def test_rows_of_many_do_not_reach_one_another(g):
    W = packed(g, 96, 512, 64, True, torch.float16, 1)
    X = torch.randn((40, 512), device=DEV).half()
    want = g.linear_w4(X, *W, group=64)
    X[5, 100], X[37, 0] = float("inf"), float("nan")
    got = g.linear_w4(X, *W, group=64)
    rows = [i for i in range(40) if i not in (5, 37)]
    assert torch.equal(got[rows], want[rows])
    assert not torch.isfinite(got[5]).any() and torch.isnan(got[37]).all()


@pytest.mark.parametrize("M", [8, 32, 64])
def test_two_streams_and_replays(g, M):
    """Calls on two streams at once and replayed from two graphs give what one call gives."""
    W = [packed(g, 4096, 1024, 128, False, torch.bfloat16, i) for i in range(2)]
    X = torch.randn((M, 1024), device=DEV).bfloat16()
    want = [g.linear_w4(X, *w, group=128) for w in W]
    streams = [torch.cuda.Stream() for _ in W]
    torch.cuda.synchronize()
    for _ in range(5):
        got = []
        for s, w in zip(streams, W):
            with torch.cuda.stream(s):
                got.append([g.linear_w4(X, *w, group=128) for _ in range(4)])
        torch.cuda.synchronize()
        assert all(torch.equal(c, want[i]) for i in range(2) for c in got[i])
    graphs, outs = [], []
    for s, w in zip(streams, W):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            outs.append(g.linear_w4(X, *w, group=128))
        graphs.append(graph)
    for _ in range(3):
        for c in outs:
            c.zero_()
        torch.cuda.synchronize()
        for s, graph in zip(streams, graphs):
            with torch.cuda.stream(s):
                graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(c, w) for c, w in zip(outs, want))
    assert g.check() == g.GEMM_OK


@pytest.mark.parametrize("N,K", [(256, 1024), (4096, 4096), (33, 64)])
def test_wait_runs_out_and_context_survives(g, N, K):
    W = packed(g, N, K, 64, True, torch.float16, 2)
    X = torch.randn((40, K), device=DEV).half()
    C = torch.full((40, N), 5.0, device=DEV).half()
    assert g.check() == g.GEMM_OK
    args = (X.data_ptr(), g.TYPES[X.dtype], W[0].data_ptr(), W[1].data_ptr(), W[2].data_ptr(), C.data_ptr(), 40, N, K, 64)
    st = g.lib().linear_w4_selftest_timeout(*args, 1 << 20, torch.cuda.current_stream().cuda_stream)
    assert st == g.GEMM_OK
    assert g.check() == g.GEMM_ERR_TIMEOUT
    assert (g.last_timeout_record() & 0xFF) == 3, hex(g.last_timeout_record())
    assert (C == 5.0).all()
    check(g, X, W, N, 64, False)
    assert g.lib().linear_w4_selftest_timeout(*args, 1, None) == g.GEMM_ERR_INVALID_ARG
    few = args[:6] + (32,) + args[7:]
    assert g.lib().linear_w4_selftest_timeout(*few, 1 << 20, None) == g.GEMM_ERR_INVALID_ARG


@pytest.mark.parametrize("xt", ["fp16", "bf16"])
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("M,N,K", [(17, 4096, 4096), (32, 16400, 1024), (24, 8200, 2056), (31, 65600, 256), (20, 130, 131072),
                                   (32, 140000, 120)])
def test_some_rows_beside_a_large_weight(g, M, N, K, group, xt):
    W = packed(g, N, K, group, group == 64, DTYPES[xt], M + N + K)
    gen = torch.Generator().manual_seed(K)
    X = torch.randn((M, K), generator=gen).to(DTYPES[xt]).to(DEV)
    C = check(g, X, W, N, group, relu=M % 2 == 0)
    buf = torch.full((M * N + 64,), 7.0, dtype=X.dtype, device=DEV)
    out = buf[32:32 + M * N].reshape(M, N)
    assert torch.equal(g.linear_w4(X, *W, N=N, group=group, relu=M % 2 == 0, C=out), C)
    assert (buf[:32] == 7).all() and (buf[32 + M * N:] == 7).all()
