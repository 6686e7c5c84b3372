"""The operators around a feed-forward block as they are used together: trained with
RMS norm and dropout, served in FP8 and with 4-bit weights."""
from __future__ import annotations

import pytest
import torch

import feed_forward_reference as ref

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda:0")
U = 2.0 ** -24


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


def rms64(h, gamma, eps):
    return h / torch.sqrt(h.square().mean(-1, keepdim=True) + eps) * gamma


def mask64(n, p, seed, offset):
    return ref.kept(0, n, p, seed, offset).double().to(DEV) / (1 - p)


# ---------------------------------------------------------------- gradients


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16, torch.float32])
def test_norm_and_dropout_gradients(ff, dtype):
    """One step of a stream: (y, h) = norm(u + s), o = h + dropout(y w), all gradients against 64 bits."""
    ag = ff.ag
    gen = torch.Generator().manual_seed(1)
    u, s, w, c1, c2 = (torch.randn((12, 264), generator=gen).to(dtype).to(DEV) for _ in range(5))
    gamma = (1 + 0.1 * torch.randn(264, generator=gen)).to(dtype).to(DEV)
    leaves = [t.clone().requires_grad_() for t in (u, s, gamma, w)]
    y, h = ag.rms_norm(leaves[0], leaves[2], 1e-5, residual=leaves[1])
    o = ag.dropout(y * leaves[3], 0.25, 7, 3, residual=h)
    ((o * c1).sum() + (h * c2).sum()).backward()
    wide = [t.detach().double().requires_grad_() for t in (u, s, gamma, w)]
    hd = wide[0] + wide[1]
    yd = rms64(hd, wide[2], 1e-5)
    od = hd + yd * wide[3] * mask64(12 * 264, 0.25, 7, 3).reshape(12, 264)
    ((od * c1.double()).sum() + (hd * c2.double()).sum()).backward()
    step = torch.finfo(dtype).eps / 2
    for got, want in zip(leaves, wide):
        # about eight chained roundings to the type of quantities of the gradient's size
        err = (got.grad.double() - want.grad).square().mean().sqrt()
        assert err <= (8 * step + 40 * U) * want.grad.square().mean().sqrt()
    assert ff.g.check() == ff.g.GEMM_OK


def test_gradients_where_only_some_are_wanted(ff):
    ag = ff.ag
    x, r = data(5, 64, 1), data(5, 64, 2)
    gamma = torch.ones(64, device=DEV).half()
    # the stream alone is used
    a, b, w = x.clone().requires_grad_(), r.clone().requires_grad_(), gamma.clone().requires_grad_()
    _, h = ag.rms_norm(a, w, residual=b)
    h.sum().backward()
    assert (a.grad == 1).all() and (b.grad == 1).all() and (w.grad == 0).all()
    # the norm alone, with respect to one of its inputs
    a = x.clone().requires_grad_()
    y, _ = ag.rms_norm(a, gamma, residual=r)
    y.sum().backward()
    want, _ = ff.g.rms_norm_bwd(torch.ones_like(x), ff.g.rms_norm_fwd(x, gamma, residual=r)[1],
                                ff.g.rms_norm_fwd(x, gamma, residual=r)[2], gamma)
    assert torch.equal(a.grad, want)
    # both inputs the same tensor: its gradient counts twice
    a = x.clone().requires_grad_()
    y, _ = ag.rms_norm(a, gamma, residual=a)
    y.sum().backward()
    h, rstd = ff.g.rms_norm_fwd(x, gamma, residual=x)[1:]
    one, _ = ff.g.rms_norm_bwd(torch.ones_like(x), h, rstd, gamma)
    assert torch.equal(a.grad, (one.float() * 2).half())
    # the residual of a dropout alone
    b = r.clone().requires_grad_()
    ag.dropout(x, 0.5, 1, residual=b).sum().backward()
    assert (b.grad == 1).all()


def test_gradients_of_strided_inputs_and_outputs(ff):
    ag = ff.ag
    base = data(96, 40, 5)
    x = base.t().clone().t().requires_grad_()   # column-major
    y = ag.rms_norm(x, residual=base)[0]
    ag.dropout(y.t(), 0.5, 3).t().square().sum().backward()
    z = base.clone().requires_grad_()
    y = ag.rms_norm(z, residual=base)[0]
    ag.dropout(y.t().contiguous(), 0.5, 3).t().square().sum().backward()
    assert torch.equal(x.grad, z.grad)


def test_changed_offset_is_an_error_and_not_another_mask(ff):
    x = data(4, 64).requires_grad_()
    off = torch.zeros(1, dtype=torch.int64, device=DEV)
    y = ff.ag.dropout(x, 0.5, 1, off)
    off.add_(1)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        y.sum().backward()


# ---------------------------------------------------------------- training


def test_layer_gradients_match_64_bits(ff):
    layer = ff.FeedForward(64, 128, device=DEV, norm="rms", dropout=0.2, seed=5)
    layer.offset.fill_(9)
    x, target = data(96, 64, 1), data(96, 64, 2)
    ((layer(x).float() - target.float()).square().mean() * 1024).backward()
    params = [layer.gamma, layer.w1, layer.w2]
    assert len(list(layer.parameters())) == 3
    wide = [p.detach().double().requires_grad_() for p in params]
    xd = x.double()
    # The ReLU's gradient is defined by the stored fp16 activation.
    with torch.no_grad():
        h16, _, _ = ff.g.rms_norm_fwd(x, layer.gamma.detach(), eps=layer.eps)
        relu = (ff.g.gemm_f16(h16, layer.w1.detach(), relu=True) > 0).double()
    u = ((rms64(xd, wide[0], layer.eps) @ wide[1]) * relu) @ wide[2]
    y = xd + u * mask64(96 * 64, 0.2, 5, 9).reshape(96, 64)
    ((y - target.double()).square().mean() * 1024).backward()
    for p, want in zip(params, wide):
        # about seven chained roundings to fp16 (2^-11 each) of quantities of the gradient's size
        err = (p.grad.double() - want.grad).square().mean().sqrt()
        assert err <= 7 * 2.0 ** -11 * want.grad.square().mean().sqrt()


@pytest.mark.parametrize("norm", ["layer", "rms"])
def test_stack_is_its_layers_one_after_another(ff, norm):
    stack = ff.FeedForwardStack(3, 64, 128, device=DEV, norm=norm, seed=2)
    x = data(40, 64)
    y = stack(x)
    want = x
    for layer in stack.layers:
        want = layer(want)
    assert torch.equal(y, want)   # the same sums, rounded alike
    y.sum().backward()
    got = [p.grad.clone() for p in stack.parameters()]
    stack.zero_grad()
    want.sum().backward()
    for a, b in zip(got, (p.grad for p in stack.parameters())):
        # dH is added before the gradient is rounded instead of after
        assert (a.double() - b.double()).square().mean().sqrt() <= 8 * 2.0 ** -11 * b.double().square().mean().sqrt()


def test_training_draws_a_new_mask_every_step(ff):
    stack = ff.FeedForwardStack(2, 64, 128, device=DEV, norm="rms", dropout=0.3)
    x = data(32, 64)
    first = stack(x)
    assert torch.equal(stack(x), first)
    losses = ff.train(stack, x, data(32, 64, 4), 3)
    assert len(losses) == 3 and all(int(layer.offset) == 3 for layer in stack.layers)
    with torch.no_grad():
        before = stack(x)
        ff.advance_dropout(stack)
        assert not torch.equal(stack(x), before)
        stack.eval()
        a = stack(x)
        ff.advance_dropout(stack)
        assert torch.equal(stack(x), a)
    assert "layers.0.offset" in stack.state_dict() and "offset" not in ff.FeedForward(8, 8, device=DEV).state_dict()


def test_captured_training_step_draws_a_new_mask_at_every_replay(ff):
    stack = ff.FeedForwardStack(2, 64, 128, device=DEV, norm="rms", dropout=0.3)
    x, target = data(32, 64, 1), data(32, 64, 2)

    def step():
        stack.zero_grad(set_to_none=True)
        ((stack(x).float() - target.float()).square().mean() * 1024).backward()
        with torch.no_grad():
            ff.advance_dropout(stack)

    want = []
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for _ in range(3):
            step()
            want.append([p.grad.clone() for p in stack.parameters()])
    torch.cuda.current_stream().wait_stream(side)
    for layer in stack.layers:
        layer.offset.zero_()
    stack.zero_grad(set_to_none=True)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for grads in want:
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(p.grad, w) for p, w in zip(stack.parameters(), grads))
    assert not torch.equal(want[0][0], want[1][0])


# ---------------------------------------------------------------- serving


@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("pow2", [False, True])
@pytest.mark.parametrize("norm", ["layer", "rms"])
@pytest.mark.parametrize("rows", [1, 70])
def test_fp8_layer_is_its_operators_by_definition(ff, rows, norm, pow2, residual):
    g = ff.g
    layer = ff.FeedForward(144, 272, device=DEV, norm=norm)
    with torch.no_grad():
        layer.gamma.copy_(1 + 0.2 * torch.randn(144, device=DEV))
    served = ff.FeedForwardFp8(layer, pow2=pow2)
    x = data(rows, 144)
    r = data(rows, 144, 8) if residual else None
    update, stream = served.branch(x, r)
    assert torch.equal(stream, x if r is None else x + r)
    assert torch.equal(served(x, r), stream + update)

    def values(q, s, block):
        s = torch.exp2(s.double() - 127) if pow2 else s.double()
        return q.float().double() * ref.spread(s, block, *q.shape)

    def product(a, w, relu):
        want = values(*a, 1) @ values(*w, 128).t()
        # up to 272 products in fp32 and one rounding to fp16
        tol = 300 * 2 * U * (values(*a, 1).abs() @ values(*w, 128).abs().t()) + 2.0 ** -11 * want.abs() + 2.0 ** -25
        return want.clamp(min=0) if relu else want, tol

    if norm == "rms":
        q = g.rms_norm_fp8(x, served.gamma, residual=r, eps=layer.eps, pow2=pow2)[:2]
    else:
        q = g.fp8_quantize(g.layer_norm_fwd(stream, served.gamma, served.beta, eps=layer.eps)[0], pow2=pow2)
    gemm = g.gemm_mxfp8_block_scaled if pow2 else g.gemm_fp8_block_scaled
    a = gemm(*q, *served.w1, relu=True)
    want, tol = product(q, served.w1, True)
    assert ((a.double() - want).abs() <= tol).all()
    want, tol = product(g.fp8_quantize(a, pow2=pow2), served.w2, False)
    assert ((update.double() - want).abs() <= tol).all()
    assert g.check() == g.GEMM_OK


@pytest.mark.parametrize("zeros", [False, True])
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("rows", [1, 9, 64])
def test_w4_layer_is_its_operators_by_definition(ff, rows, group, zeros):
    layer = ff.FeedForward(136, 264, device=DEV, norm="rms")
    served = ff.FeedForwardW4(layer, group=group, zeros=zeros)
    x, r = data(rows, 136), data(rows, 136, 8)
    update, stream = served.branch(x, r)
    w1 = ref.weight_w4(*served.w1, 264, 136, group)
    w2 = ref.weight_w4(*served.w2, 136, 264, group)
    h = ff.g.rms_norm_fwd(x, served.gamma, residual=r, eps=layer.eps)[0].double()
    a = ff.g.linear_w4(h.half(), *served.w1, N=264, group=group, relu=True)
    for got, inp, w, relu in ((a, h, w1, True), (update, a.double(), w2, False)):
        want = inp @ w.t()
        # as in the product's own tests
        tol = 500 * U * (inp.abs() @ w.abs().t()) + 2.0 ** -11 * want.abs() + 2.0 ** -25
        assert ((got.double() - (want.clamp(min=0) if relu else want)).abs() <= tol).all()
    with pytest.raises(ValueError):
        served(data(65, 136))


@pytest.mark.parametrize("kind", ["mxfp4", "fp8", "w4"])
@pytest.mark.parametrize("norm", ["layer", "rms"])
def test_served_stack_adds_the_updates_in_its_norms(ff, kind, norm):
    stack = ff.FeedForwardStack(3, 128, 256, device=DEV, norm=norm)
    layers = [ff.SERVED[kind](layer) for layer in stack.layers]
    x = data(7, 128)
    want = x
    for layer in layers:
        want = layer(want)
    assert torch.equal(ff.serve(stack, kind)(x), want)


@pytest.mark.parametrize("kind", ["mxfp4", "fp8", "w4"])
def test_decoding_step_in_a_graph(ff, kind):
    stack = ff.FeedForwardStack(2, 256, 512, device=DEV, norm="rms")
    served = ff.serve(stack, kind)
    x = data(1, 256)
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


@pytest.mark.parametrize("kind", ["mxfp4", "fp8", "w4"])
def test_command_runs(ff, capsys, kind):
    ff.main(["--rows", "64", "--dim", "128", "--hidden", "256", "--steps", "2", "--norm", "rms", "--dropout", "0.1",
             "--layers", "2", "--serve", kind])
    assert f'"ms_{kind}"' in capsys.readouterr().out


# ---------------------------------------------------------------- streams, two graphs, two calls


def calls(ff):
    g = ff.g
    x, r, w = data(64, 512, 1), data(64, 512, 2), data(1, 512, 3)[0]
    _, h, rstd = g.rms_norm_fwd(x, w, residual=r)
    W = g.w4_quantize(data(256, 512, 4))
    off = torch.full((1,), 5, dtype=torch.int64, device=DEV)
    return {"rms_norm_fwd": lambda s: g.rms_norm_fwd(x, w, residual=r, stream=s),
            "rms_norm_fp8": lambda s: g.rms_norm_fp8(x, w, residual=r, stream=s),
            "rms_norm_bwd": lambda s: g.rms_norm_bwd(r, h, rstd, w, dH=x, stream=s),
            "fp8_quantize": lambda s: g.fp8_quantize(x, stream=s),
            "dropout": lambda s: (g.dropout(x, 0.5, 3, off, residual=r, stream=s),),
            "w4_quantize": lambda s: g.w4_quantize(x, zeros=True, stream=s),
            "linear_w4": lambda s: (g.linear_w4(x, *W, stream=s),)}


NAMES = ["rms_norm_fwd", "rms_norm_fp8", "rms_norm_bwd", "fp8_quantize", "dropout", "w4_quantize", "linear_w4"]


@pytest.mark.parametrize("name", NAMES)
def test_pending_work_on_the_current_stream_does_not_reach_the_outputs(ff, name):
    call = calls(ff)[name]
    want = call(None)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    torch.cuda.empty_cache()
    # blocks of the outputs' sizes, freed with a fill still queued behind some 10 ms
    blocks = [torch.empty_like(t) for t in want]
    torch.cuda._sleep(20_000_000)
    for t in blocks:
        t.view(torch.uint8).fill_(0x55)
    del blocks, t
    got = call(side)
    torch.cuda.synchronize()
    assert ff.g.check() == ff.g.GEMM_OK
    for a, b in zip(got, want):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))


@pytest.mark.parametrize("name", [n for n in NAMES if n != "w4_quantize"])
def test_short_and_long_way_give_the_same(ff, monkeypatch, name):
    g = ff.g
    call = calls(ff)[name]
    g._short()
    with monkeypatch.context() as m:
        m.setattr(g, "_call", None)   # the long way's last step
        got = call(None)
    with monkeypatch.context() as m:
        import types
        never = {n: lambda *a: None for n in ("rms_norm_fwd", "rms_norm_fp8", "rms_norm_bwd", "fp8_quantize", "dropout",
                                              "linear_w4")}
        m.setattr(g, "_binding", types.SimpleNamespace(**never))
        want = call(None)
    assert len(got) == len(want)
    for a, b in zip(got, want):
        assert a.dtype == b.dtype and a.stride() == b.stride() and a.device == b.device
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))


def test_short_way_leaves_anything_else_to_the_long_way(ff):
    g = ff.g
    b = g._short()
    assert b.torch_version == torch.__version__
    x, w = data(4, 128), data(1, 128)[0]
    r = torch.ones(4, device=DEV)
    Q, S, Z = g.w4_quantize(data(32, 128), zeros=True)
    off = torch.zeros(1, dtype=torch.int64, device=DEV)
    plain = {"rms_norm_fwd": (x, w, x, 1e-6, True), "rms_norm_fp8": (x, w, x, 1e-6, False),
             "rms_norm_bwd": (x, x, r, w, x, True), "fp8_quantize": (x, 1, False), "dropout": (x, 0.5, 1, off, x),
             "linear_w4": (x, Q, S, Z, 32, 128, False)}
    for name, args in plain.items():
        assert getattr(b, name)(*args) is not None
        for i, a in enumerate(args):
            if isinstance(a, torch.Tensor):
                others = [a.cpu(), a.double() if a.is_floating_point() else a.int(), a[:0], [1], torch.stack([a, a])]
                if a.dim() > 1:
                    others += [a.transpose(0, 1), a[:1] if name != "linear_w4" or i else a[:, :64]]
                if i == 0 or (name == "rms_norm_bwd" and i == 1):
                    # another type, size or shape of the input alone is another call's plain one
                    others = others[:2] + others[3:4] + ([a.transpose(0, 1)] if a.dim() > 1 else [])
            elif isinstance(a, float):
                others = ["a"] if name != "dropout" else ["a", 1.0, -0.1, float("nan")]
            elif isinstance(a, bool):
                continue
            else:
                others = ["a", -1]
            for o in others:
                got = getattr(b, name)(*args[:i], o, *args[i + 1:])
                assert got is None, (name, i, o)
    assert b.linear_w4(x, Q, S, Z, 33, 128, False) is None and b.linear_w4(x, Q, S, Z, 32, 64, False) is None
    assert b.fp8_quantize(x, 64, False) is None
    assert b.dropout(x, 0.5, 1 << 64, 0, None) is None and b.dropout(x, 0.5, 1, -1, None) is None
    with pytest.raises(ValueError):
        g.dropout(x, 0.5, 1 << 64)
    assert g.check() == g.GEMM_OK


@pytest.mark.parametrize("name", NAMES)
def test_calls_on_two_streams_at_once(ff, name):
    call = calls(ff)[name]
    want = call(None)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [[call(s) for s in streams] for _ in range(8)]
    torch.cuda.synchronize()
    for pair in got:
        for out in pair:
            for a, b in zip(out, want):
                assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))


def test_host_tensors_are_refused(ff):
    g = ff.g
    x = torch.zeros((4, 128), dtype=torch.float16)
    side = torch.cuda.Stream()
    W = g.w4_pack(torch.zeros((16, 128), dtype=torch.uint8), torch.zeros((16, 1), dtype=torch.float16))
    for call in (lambda s: g.rms_norm_fwd(x, stream=s), lambda s: g.rms_norm_fp8(x, stream=s),
                 lambda s: g.rms_norm_bwd(x, x, torch.zeros(4), weights=False, stream=s),
                 lambda s: g.fp8_quantize(x, stream=s), lambda s: g.dropout(x, 0.5, 1, stream=s),
                 lambda s: g.w4_quantize(x, stream=s), lambda s: g.linear_w4(x, *W, stream=s)):
        with pytest.raises((g.GemmError, ValueError)):
            call(side)
    assert g.check() == g.GEMM_OK
