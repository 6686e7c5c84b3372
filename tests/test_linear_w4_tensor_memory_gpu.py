"""GPU tests of the tensor memory kernel of products with 4-bit weights: waits that run
out, streams and replays, and what lies beside X."""
from __future__ import annotations

import pytest
import torch

from test_linear_w4_gpu import DEV, DTYPES, check, g, packed  # noqa: F401  (g: a fixture)

pytestmark = pytest.mark.gpu


def give_up(g, hook, X, W, C, group):
    """One launch whose last block of K's share never gets W; its status and the site where a wait ran out."""
    M, K = X.shape
    assert g.check() == g.GEMM_OK
    st = hook(X.data_ptr(), g.TYPES[X.dtype], W[0].data_ptr(), W[1].data_ptr(), W[2].data_ptr() if W[2] is not None else None,
              C.data_ptr(), M, C.shape[1], K, group, 1 << 20, torch.cuda.current_stream().cuda_stream)
    assert st == g.GEMM_OK
    assert g.check() == g.GEMM_ERR_TIMEOUT
    return g.last_timeout_record() & 0xFF


# K by itself, and over two, four and eight blocks.
@pytest.mark.parametrize("N,K", [(20000, 1024), (9728, 1024), (4096, 2048), (256, 1024), (256, 4096), (130, 16384)])
def test_no_block_of_a_cluster_stores_where_one_gave_up(g, N, K):  # noqa: F811
    W = packed(g, N, K, 64, True, torch.float16, 3)
    X = torch.randn((64, K), device=DEV).half()
    C = torch.full((64, N), 5.0, device=DEV).half()
    assert give_up(g, g.lib().linear_w4_selftest_timeout, X, W, C, 64) == 3
    assert (C == 5.0).all()
    check(g, X, W, N, 64, False)


# The kernel for up to 32 rows: K by itself, over two, and over more blocks of a cluster.
@pytest.mark.parametrize("group,zeros", [(32, True), (64, False), (128, True)])
@pytest.mark.parametrize("M,N,K", [(32, 4096, 4096), (17, 16400, 1024), (24, 2048, 8192), (20, 130, 131072)])
def test_waits_of_the_kernel_for_few_rows_run_out(g, M, N, K, group, zeros):  # noqa: F811
    W = packed(g, N, K, group, zeros, torch.bfloat16, 2)
    X = torch.randn((M, K), device=DEV).bfloat16()
    C = torch.full((M, N), 5.0, device=DEV).bfloat16()
    assert give_up(g, g.lib().linear_w4_few_selftest_timeout, X, W, C, group) == 3
    assert (C == 5.0).all()
    check(g, X, W, N, group, False)


def test_the_few_rows_hook_refuses_what_another_kernel_takes(g):  # noqa: F811
    L, bad = g.lib(), g.GEMM_ERR_INVALID_ARG
    for M, N, K in ((16, 4096, 4096), (32, 4096, 4095), (32, 4095, 4096), (33, 4096, 4096), (32, 0, 4096), (32, 4096, 0)):
        assert L.linear_w4_few_selftest_timeout(16, 0, 16, 16, None, 16, M, N, K, 64, 1 << 20, None) == bad
    assert L.linear_w4_few_selftest_timeout(16, 0, 16, 16, None, 16, 32, 4096, 4096, 64, 1, None) == bad


@pytest.mark.parametrize("xt", ["fp16", "bf16"])
@pytest.mark.parametrize("group,zeros", [(32, False), (32, True), (64, False), (64, True), (128, False), (128, True)])
@pytest.mark.parametrize("M,N,K", [(32, 4096, 4096), (17, 4100, 4104), (25, 1030, 16384)])
def test_few_rows_with_and_without_zero_points(g, M, N, K, group, zeros, xt):  # noqa: F811
    """X among NaNs, on the 16-byte grid and off it; C among other numbers."""
    W = packed(g, N, K, group, zeros, DTYPES[xt], M + N + K)
    gen = torch.Generator().manual_seed(K)
    X = torch.randn((M, K), generator=gen).to(DTYPES[xt]).to(DEV)
    C = check(g, X, W, N, group, relu=M % 2 == 0)
    for by in (8, 3):
        flat = torch.full((M * K + 16,), float("nan"), dtype=X.dtype, device=DEV)
        flat[by:by + M * K].copy_(X.reshape(-1))
        buf = torch.full((M * N + 64,), 7.0, dtype=X.dtype, device=DEV)
        out = buf[32:32 + M * N].reshape(M, N)
        got = g.linear_w4(flat[by:by + M * K].reshape(M, K), *W, N=N, group=group, relu=M % 2 == 0, C=out)
        assert torch.equal(got, C)
        assert (buf[:32] == 7).all() and (buf[32 + M * N:] == 7).all()


@pytest.mark.parametrize("M", [17, 32])
def test_rows_of_few_do_not_reach_one_another(g, M):  # noqa: F811
    W = packed(g, 4096, 4096, 64, True, torch.float16, 1)
    X = torch.randn((M, 4096), device=DEV).half()
    want = g.linear_w4(X, *W, group=64)
    X[5, 100], X[M - 1, 0], X[0, 4095] = float("inf"), float("nan"), float("-inf")
    got = g.linear_w4(X, *W, group=64)
    rows = [i for i in range(M) if i not in (0, 5, M - 1)]
    assert torch.equal(got[rows], want[rows])
    # inf (q - z) s with q = z is NaN, so no element of such a row is finite
    assert not torch.isfinite(got[[0, 5]]).any() and torch.isnan(got[M - 1]).all()


@pytest.mark.parametrize("M,N,K", [(32, 4096, 4096), (20, 1024, 16384)])
def test_two_streams_and_replays_of_few_rows(g, M, N, K):  # noqa: F811
    """Calls on two streams at once and replayed from two graphs give what one call gives."""
    W = [packed(g, N, K, 128, i == 1, torch.bfloat16, i) for i in range(2)]
    X = torch.randn((M, K), device=DEV).bfloat16()
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
            outs.append([g.linear_w4(X, *w, group=128) for _ in range(3)])
        graphs.append(graph)
    for _ in range(3):
        for c in outs[0] + outs[1]:
            c.zero_()
        torch.cuda.synchronize()
        for s, graph in zip(streams, graphs):
            with torch.cuda.stream(s):
                graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(c, want[i]) for i in range(2) for c in outs[i])
    assert g.check() == g.GEMM_OK
