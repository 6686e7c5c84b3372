"""The feed-forward example: the new operators together, trained and served."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import mxfp4_reference as ref

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda:0")


@pytest.fixture(scope="module")
def ff():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    from dense_fp16_gemm_05_gb300 import build as gbuild
    gbuild.build()
    from dense_fp16_gemm_05_gb300 import feed_forward
    return feed_forward


def data(rows, dim, seed=3):
    gen = torch.Generator().manual_seed(seed)
    return torch.randn((rows, dim), generator=gen).half().to(DEV)


@pytest.mark.parametrize("rows", [1, 5, 200])
def test_served_layer_is_its_operators_by_definition(ff, rows):
    g = ff.g
    layer = ff.FeedForward(136, 264, device=DEV)
    served = ff.FeedForwardMxfp4(layer)
    x = data(rows, 136)
    got = served(x)
    # each stage on the kernel's own input: quantisation exactly, products to the tolerance
    h, _, _ = g.layer_norm_fwd(x, layer.gamma.detach(), layer.beta.detach(), eps=layer.eps)
    w1 = ref.decode(*ref.quantize(layer.w1.detach().t().cpu().double().numpy()))[:, :136]
    w2 = ref.decode(*ref.quantize(layer.w2.detach().t().cpu().double().numpy()))[:, :264]
    qa = ref.decode(*ref.quantize(h.cpu().double().numpy()))[:, :136]
    a = g.gemm_mxfp4(*g.mxfp4_quantize(h), *served.w1, relu=True, K=136)
    want, mag = ref.product(qa, w1, True)
    assert np.all(np.abs(a.cpu().double().numpy() - want) <= ref.product_tolerance(want, mag, 136))
    qb = ref.decode(*ref.quantize(a.cpu().double().numpy()))[:, :264]
    want, mag = ref.product(qb, w2, False)
    y = (got.cpu().double() - x.cpu().double()).numpy()
    # the sum with x rounds once more to fp16: half a step of the result, 2^-11 relative
    tol = ref.product_tolerance(want, mag, 264) + 2.0 ** -11 * np.abs(got.cpu().double().numpy()) + 2.0 ** -25
    assert np.all(np.abs(y - want) <= 1.01 * tol)


def test_training_lowers_the_loss_and_gradients_match_fp64(ff):
    layer = ff.FeedForward(64, 128, device=DEV)
    x, target = data(96, 64, 1), data(96, 64, 2)
    layer.zero_grad()
    loss = (layer(x).float() - target.float()).square().mean()
    (loss * 1024).backward()
    leaves = [p.detach().double().requires_grad_() for p in (layer.gamma, layer.beta, layer.w1, layer.w2)]
    xd = x.double()
    mean = xd.mean(-1, keepdim=True)
    z = (xd - mean) / torch.sqrt((xd - mean).square().mean(-1, keepdim=True) + layer.eps)
    # The ReLU's gradient is defined by the stored fp16 activation (see
    # gemm_f16_relu_backward): an element that rounding moved across zero is on
    # the side where the layer has it.
    with torch.no_grad():
        h16, _, _ = ff.g.layer_norm_fwd(x, layer.gamma.detach(), layer.beta.detach(), eps=layer.eps)
        mask = (ff.g.gemm_f16(h16, layer.w1.detach(), relu=True) > 0).double()
    y = xd + (((z * leaves[0] + leaves[1]) @ leaves[2]) * mask) @ leaves[3]
    ((y - target.double()).square().mean() * 1024).backward()
    for p, want in zip((layer.gamma, layer.beta, layer.w1, layer.w2), leaves):
        # about six chained roundings to fp16 (2^-11 each) of quantities of the gradient's size
        err = (p.grad.double() - want.grad).square().mean().sqrt()
        assert err <= 6 * 2.0 ** -11 * want.grad.square().mean().sqrt()
    losses = ff.train(layer, x, target, 5)
    assert losses[-1] < losses[0]


def test_decoding_step_in_a_graph(ff):
    layer = ff.FeedForward(256, 512, device=DEV)
    served = ff.FeedForwardMxfp4(layer)
    x = data(1, 256)
    want = served(x)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        served(x)
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = served(x)
    for seed in (3, 4):
        x.copy_(data(1, 256, seed))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, served(x))
    x.copy_(data(1, 256))
    assert torch.equal(served(x), want)


def test_command_runs(ff, capsys):
    ff.main(["--rows", "64", "--dim", "128", "--hidden", "256", "--steps", "2"])
    assert '"ms_mxfp4"' in capsys.readouterr().out


def test_training_step_in_a_graph(ff):
    # forward and backward captured together, after warm-up on a side stream and
    # with no eager graph of the parameters alive
    layer = ff.FeedForward(128, 256, device=DEV)
    x, target = data(64, 128, 1), data(64, 128, 2)

    def step():
        layer.zero_grad(set_to_none=True)
        loss = (layer(x).float() - target.float()).square().mean() * 1024.0
        loss.backward()

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for _ in range(2):
            step()
    torch.cuda.current_stream().wait_stream(side)
    want = [p.grad.clone() for p in layer.parameters()]
    layer.zero_grad(set_to_none=True)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for _ in range(2):
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(p.grad, w) for p, w in zip(layer.parameters(), want))


@pytest.mark.parametrize("relu", [False, True])
@pytest.mark.parametrize("M,N,K", [(1, 8, 8), (40, 24, 72), (130, 264, 136), (257, 128, 320)])
def test_four_bit_linear_and_its_gradients(ff, M, N, K, relu):
    ag, g = ff.ag, ff.g
    gen = torch.Generator().manual_seed(M + N + K)
    A = torch.randn((M, K), generator=gen).half().to(DEV).requires_grad_()
    B = torch.randn((K, N), generator=gen).half().to(DEV).requires_grad_()
    dC = torch.randn((M, N), generator=gen).half().to(DEV)
    C = ag.linear_mxfp4(A, B, relu)
    C.backward(dC)
    a = ref.decode(*ref.quantize(A.detach().cpu().double().numpy()))[:, :K]
    b = ref.decode(*ref.quantize(B.detach().t().cpu().double().numpy()))[:, :K]      # (N,K)
    want, mag = ref.product(a, b, relu)
    assert np.all(np.abs(C.detach().cpu().double().numpy() - want) <= ref.product_tolerance(want, mag, K))
    # the linear map of the quantised values, with the mask of the stored output
    dz = dC.cpu().double().numpy() * ((C.detach() > 0).cpu().numpy() if relu else 1.0)
    for got, x, y in ((A.grad, dz, b), (B.grad, a.T, dz)):
        want = x @ y
        # one rounding to fp16, and fp32 sums of up to 320 exact products
        tol = 2.0 ** -11 * np.abs(want) + 2.0 ** -25 + 330 * 2.0 ** -24 * (np.abs(x) @ np.abs(y))
        assert np.all(np.abs(got.cpu().double().numpy() - want) <= tol)


def test_four_bit_gradients_only_where_wanted(ff):
    A, B = data(16, 64, 1), data(64, 32, 2).requires_grad_()
    ff.ag.linear_mxfp4(A, B).sum().backward()
    assert A.grad is None and B.grad.shape == (64, 32)


def test_four_bit_training_matches_the_served_layer(ff):
    layer = ff.FeedForward(64, 128, device=DEV, four_bit=True)
    x, target = data(96, 64, 1), data(96, 64, 2)
    losses = ff.train(layer, x, target, 5)
    assert losses[-1] < losses[0]
    with torch.no_grad():
        assert torch.equal(layer(x), ff.FeedForwardMxfp4(layer)(x))   # the same kernels on the same codes
