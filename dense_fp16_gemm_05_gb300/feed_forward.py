"""A pre-norm feed-forward layer on the library's kernels: trained in fp16, served in 4 bits or FP8.

    python -m dense_fp16_gemm_05_gb300.feed_forward [--rows 4096 --dim 1024 --hidden 4096 --steps 3] [--four-bit]
        [--norm layer|rms] [--dropout 0.1] [--layers 2] [--serve mxfp4|fp8|w4]

:class:`FeedForward` is y = x + ReLU(norm(x) @ W1) @ W2 with layer norm or RMS norm,
the fp16 GEMMs and their gradients (``autograd``), with ``dropout`` on what is added
to x, or, with ``four_bit``, 4-bit products trained straight through the
quantisation; :class:`FeedForwardStack` is several, each adding the one before in
its norm.  For inference :class:`FeedForwardMxfp4` quantises the activations in front
of either product to MXFP4, :class:`FeedForwardFp8` to FP8 (prompts; the norm
itself writes FP8), and :class:`FeedForwardW4` keeps 16-bit activations beside 4-bit
weights (a few rows: tokens being generated); their weights are quantised once.
The command trains layers for a few steps, converts them and prints both forms'
times and how far the served output is from the trained one's (nothing, with
--four-bit).
"""
from __future__ import annotations

import argparse
import json

import torch

from . import autograd as ag
from . import gemm_f16 as g


class FeedForward(torch.nn.Module):
    """x + ReLU(norm(x) @ W1) @ W2 on fp16 CUDA tensors (rows, dim); dim and hidden multiples of 8.

    ``norm`` is "layer" or "rms" (without a beta).  With ``dropout`` > 0, in training
    mode, the branch's elements are dropped before they are added to x; the mask is a
    function of ``seed`` and the layer's ``offset``, an int64 tensor that a training
    step advances after its backward pass (``train`` does; inside a captured step too).
    """

    def __init__(self, dim: int, hidden: int, eps: float = 1e-5, device="cuda:0", seed: int = 0,
                 four_bit: bool = False, norm: str = "layer", dropout: float = 0.0):
        super().__init__()
        if norm not in ("layer", "rms"):
            raise ValueError(f"norm must be 'layer' or 'rms', got {norm!r}")
        if not 0.0 <= dropout < 1.0:
            raise ValueError(f"dropout must be in [0, 1), got {dropout}")
        self.four_bit, self.norm, self.dropout, self.seed = four_bit, norm, dropout, seed
        gen = torch.Generator(device="cpu").manual_seed(seed)
        self.eps = eps
        self.gamma = torch.nn.Parameter(torch.ones(dim, dtype=torch.float16, device=device))
        self.beta = None
        if norm == "layer":
            self.beta = torch.nn.Parameter(torch.zeros(dim, dtype=torch.float16, device=device))
        w1 = torch.randn((dim, hidden), generator=gen) * (2.0 / dim) ** 0.5
        w2 = torch.randn((hidden, dim), generator=gen) * (1.0 / hidden) ** 0.5
        self.w1 = torch.nn.Parameter(w1.half().to(device))
        self.w2 = torch.nn.Parameter(w2.half().to(device))
        if dropout > 0.0:
            self.register_buffer("offset", torch.zeros(1, dtype=torch.int64, device=device))

    def _products(self, h: torch.Tensor) -> torch.Tensor:
        if self.four_bit:
            return ag.linear_mxfp4(ag.linear_mxfp4(h, self.w1, relu=True), self.w2)
        return ag.gemm(ag.gemm_relu(h, self.w1), self.w2)

    def _drops(self) -> bool:
        return self.dropout > 0.0 and self.training

    def forward(self, x: torch.Tensor) -> torch.Tensor:
        if self.norm == "rms":
            h = ag.rms_norm(x, self.gamma, self.eps)
        else:
            h = ag.layer_norm(x, self.gamma, self.beta, self.eps)
        u = self._products(h)
        return ag.dropout(u, self.dropout, self.seed, self.offset, residual=x) if self._drops() else x + u

    def branch(self, x: torch.Tensor, residual: torch.Tensor | None = None):
        """(update, stream): what the layer adds to the stream x (+ residual), and that stream.

        The two are added by whoever comes next, a following layer's norm in its own
        kernel.
        """
        if self.norm == "rms":
            if residual is None:
                h, stream = ag.rms_norm(x, self.gamma, self.eps), x
            else:
                h, stream = ag.rms_norm(x, self.gamma, self.eps, residual=residual)
        else:
            stream = x if residual is None else x + residual
            h = ag.layer_norm(stream, self.gamma, self.beta, self.eps)
        u = self._products(h)
        return (ag.dropout(u, self.dropout, self.seed, self.offset) if self._drops() else u), stream


class FeedForwardStack(torch.nn.Module):
    """``layers`` feed-forward layers, each adding the update of the one before in its norm."""

    def __init__(self, layers: int, dim: int, hidden: int, seed: int = 0, **kw):
        super().__init__()
        if layers < 1:
            raise ValueError(f"layers must be at least 1, got {layers}")
        self.layers = torch.nn.ModuleList(FeedForward(dim, hidden, seed=seed + i, **kw) for i in range(layers))

    def forward(self, x: torch.Tensor) -> torch.Tensor:
        update = None
        for layer in self.layers:
            update, x = layer.branch(x) if update is None else layer.branch(update, x)
        return x + update


class _Served:
    """What the served forms share: copies of the norm, the residual stream.

    No gradient is recorded: the output of an input that requires one is detached
    from it (through the residual alone a gradient would be wrong).  A call takes
    x, or, with ``residual``, their sum as its input.
    """

    def __init__(self, layer: FeedForward):
        self.eps, self.norm = layer.eps, layer.norm
        # Copies, as the packed weights are: training the layer further changes neither.
        self.gamma = layer.gamma.detach().clone()
        self.beta = None if layer.beta is None else layer.beta.detach().clone()
        self.dim, self.hidden = layer.w1.shape

    def _norm(self, x: torch.Tensor, residual: torch.Tensor | None):
        """(norm, stream) of x (+ residual), both detached."""
        x = x.detach()
        if self.norm == "rms":
            h, stream, _ = g.rms_norm_fwd(x, self.gamma, residual=None if residual is None else residual.detach(),
                                          eps=self.eps, stats=False)
            return h, stream
        stream = x if residual is None else x + residual.detach()
        h, _, _ = g.layer_norm_fwd(stream, self.gamma, self.beta, eps=self.eps, stats=False)
        return h, stream

    def branch(self, x: torch.Tensor, residual: torch.Tensor | None = None):
        """(update, stream), as FeedForward.branch."""
        h, stream = self._norm(x, residual)
        return self._products(h), stream

    def __call__(self, x: torch.Tensor, residual: torch.Tensor | None = None) -> torch.Tensor:
        update, stream = self.branch(x, residual)
        return stream + update


class FeedForwardMxfp4(_Served):
    """The layer with MXFP4 weights and activations, for inference.

    The weights are stored in-features x out-features, so their columns are
    quantised (``transpose=True``): blocks of 32 along the dimension that the
    product sums over.
    """

    def __init__(self, layer: FeedForward):
        super().__init__(layer)
        self.w1 = g.mxfp4_quantize(layer.w1.detach(), transpose=True)
        self.w2 = g.mxfp4_quantize(layer.w2.detach(), transpose=True)

    def _products(self, h: torch.Tensor) -> torch.Tensor:
        a = g.gemm_mxfp4(*g.mxfp4_quantize(h), *self.w1, relu=True, K=self.dim)
        return g.gemm_mxfp4(*g.mxfp4_quantize(a), *self.w2, K=self.hidden)


class FeedForwardFp8(_Served):
    """The layer with FP8 weights (a scale per 128 x 128) and activations (per 1 x 128), for inference.

    An RMS norm writes its output in FP8 itself.  ``pow2``: power-of-two scales, which
    the tensor core applies.  dim and hidden are multiples of 16.
    """

    def __init__(self, layer: FeedForward, pow2: bool = False):
        super().__init__(layer)
        if self.dim % 16 or self.hidden % 16:
            raise ValueError(f"dim and hidden must be multiples of 16, got {self.dim} and {self.hidden}")
        self.pow2 = pow2
        # (out-features, in-features), as the products take weights.
        self.w1 = g.fp8_quantize(layer.w1.detach().t().contiguous(), block_rows=128, pow2=pow2)
        self.w2 = g.fp8_quantize(layer.w2.detach().t().contiguous(), block_rows=128, pow2=pow2)

    def _gemm(self, a, w, relu: bool) -> torch.Tensor:
        return (g.gemm_mxfp8_block_scaled if self.pow2 else g.gemm_fp8_block_scaled)(*a, *w, relu=relu)

    def branch(self, x: torch.Tensor, residual: torch.Tensor | None = None):
        if self.norm == "rms":
            q, s, stream = g.rms_norm_fp8(x.detach(), self.gamma, residual=None if residual is None else residual.detach(),
                                          eps=self.eps, pow2=self.pow2)
        else:
            h, stream = self._norm(x, residual)
            q, s = g.fp8_quantize(h, pow2=self.pow2)
        a = self._gemm((q, s), self.w1, True)
        return self._gemm(g.fp8_quantize(a, pow2=self.pow2), self.w2, False), stream


class FeedForwardW4(_Served):
    """The layer with 4-bit weights (a scale per ``group`` input features) beside fp16 activations, for
    at most 64 rows at a time: tokens being generated."""

    def __init__(self, layer: FeedForward, group: int = 128, zeros: bool = False):
        super().__init__(layer)
        self.group = group
        self.w1 = g.w4_quantize(layer.w1.detach(), group, zeros, transpose=True)
        self.w2 = g.w4_quantize(layer.w2.detach(), group, zeros, transpose=True)

    def _products(self, h: torch.Tensor) -> torch.Tensor:
        a = g.linear_w4(h, *self.w1, N=self.hidden, group=self.group, relu=True)
        return g.linear_w4(a, *self.w2, N=self.dim, group=self.group)


SERVED = {"mxfp4": FeedForwardMxfp4, "fp8": FeedForwardFp8, "w4": FeedForwardW4}


def serve(stack: FeedForwardStack, kind: str, **kw):
    """A function x -> y: the stack's layers in the served form ``kind``, each adding the update of the
    one before in its norm."""
    layers = [SERVED[kind](layer, **kw) for layer in stack.layers]

    def run(x: torch.Tensor) -> torch.Tensor:
        update, x = layers[0].branch(x)
        for layer in layers[1:]:
            update, x = layer.branch(update, x)
        return x + update

    return run


def advance_dropout(module: torch.nn.Module) -> None:
    """Moves every layer's dropout to its next mask; after a step's backward pass, also inside a captured step."""
    for m in module.modules():
        if isinstance(m, FeedForward) and m.dropout > 0.0:
            m.offset.add_(1)


def train(layer: torch.nn.Module, x: torch.Tensor, target: torch.Tensor, steps: int, lr: float = 0.05) -> list[float]:
    """Plain gradient steps on the mean squared error; returns the losses."""
    losses = []
    for _ in range(steps):
        layer.zero_grad(set_to_none=True)
        loss = (layer(x).float() - target.float()).square().mean()
        # The gradient is scaled up for fp16 and the step down again.
        (loss * 1024.0).backward()
        with torch.no_grad():
            for p in layer.parameters():
                p -= (lr / 1024.0) * p.grad
            advance_dropout(layer)
        losses.append(float(loss.detach()))
    return losses


def _time(fn, reps: int = 10) -> float:
    fn()
    s, e = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    best = float("inf")
    for _ in range(reps):
        s.record()
        fn()
        e.record()
        e.synchronize()
        best = min(best, s.elapsed_time(e))
    return best


def main(argv=None):
    p = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    p.add_argument("--rows", type=int, default=4096)
    p.add_argument("--dim", type=int, default=1024)
    p.add_argument("--hidden", type=int, default=4096)
    p.add_argument("--steps", type=int, default=3)
    p.add_argument("--four-bit", action="store_true", help="train with 4-bit products")
    p.add_argument("--norm", choices=["layer", "rms"], default="layer")
    p.add_argument("--dropout", type=float, default=0.0)
    p.add_argument("--layers", type=int, default=1)
    p.add_argument("--serve", choices=sorted(SERVED), default="mxfp4", help="the form served")
    args = p.parse_args(argv)
    dev = torch.device("cuda", 0)
    gen = torch.Generator(device=dev).manual_seed(1)
    x = torch.randn((args.rows, args.dim), generator=gen, device=dev).half()
    target = torch.randn((args.rows, args.dim), generator=gen, device=dev).half()
    stack = FeedForwardStack(args.layers, args.dim, args.hidden, device=dev, four_bit=args.four_bit, norm=args.norm,
                             dropout=args.dropout)
    losses = train(stack, x, target, args.steps)
    served = serve(stack, args.serve)
    stack.eval()
    if args.serve == "w4":   # a few rows
        x = x[:g.W4_MAX_ROWS].contiguous()
    with torch.no_grad():
        want, got = stack(x).float(), served(x).float()
        ms16, ms_served = _time(lambda: stack(x)), _time(lambda: served(x))
    st = g.check()
    if st != g.GEMM_OK:
        raise SystemExit(f"device status {st}: {g.strerror(st)}")
    update = (want - x.float()).square().mean().sqrt()
    print(json.dumps({"rows": x.shape[0], "dim": args.dim, "hidden": args.hidden, "layers": args.layers, "norm": args.norm,
                      "losses": losses, "ms_trained": ms16, f"ms_{args.serve}": ms_served,
                      "rms_difference_of_update": float((want - got).square().mean().sqrt() / update)}))


if __name__ == "__main__":
    main()
