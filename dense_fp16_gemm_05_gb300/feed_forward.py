"""A pre-norm feed-forward layer on the library's kernels: trained in fp16, served in 4 bits.

    python -m dense_fp16_gemm_05_gb300.feed_forward [--rows 4096 --dim 1024 --hidden 4096 --steps 3] [--four-bit]

:class:`FeedForward` is y = x + ReLU(norm(x) @ W1) @ W2 with layer norm, the
fp16 GEMMs and their gradients (``autograd``), or, with ``four_bit``, 4-bit
products trained straight through the quantisation.  :class:`FeedForwardMxfp4` is the
same layer for inference: its weights are quantised to MXFP4 once, each call
quantises the activations in front of either product.  The command trains a
layer for a few steps, converts it and prints both layers' times and how far
the served layer's output is from the trained one's (nothing, with --four-bit).
"""
from __future__ import annotations

import argparse
import json

import torch

from . import autograd as ag
from . import gemm_f16 as g


class FeedForward(torch.nn.Module):
    """x + ReLU(norm(x) @ W1) @ W2 on fp16 CUDA tensors (rows, dim); dim and hidden multiples of 8."""

    def __init__(self, dim: int, hidden: int, eps: float = 1e-5, device="cuda:0", seed: int = 0,
                 four_bit: bool = False):
        super().__init__()
        self.four_bit = four_bit
        gen = torch.Generator(device="cpu").manual_seed(seed)
        self.eps = eps
        self.gamma = torch.nn.Parameter(torch.ones(dim, dtype=torch.float16, device=device))
        self.beta = torch.nn.Parameter(torch.zeros(dim, dtype=torch.float16, device=device))
        w1 = torch.randn((dim, hidden), generator=gen) * (2.0 / dim) ** 0.5
        w2 = torch.randn((hidden, dim), generator=gen) * (1.0 / hidden) ** 0.5
        self.w1 = torch.nn.Parameter(w1.half().to(device))
        self.w2 = torch.nn.Parameter(w2.half().to(device))

    def forward(self, x: torch.Tensor) -> torch.Tensor:
        h = ag.layer_norm(x, self.gamma, self.beta, self.eps)
        if self.four_bit:
            return x + ag.linear_mxfp4(ag.linear_mxfp4(h, self.w1, relu=True), self.w2)
        return x + ag.gemm(ag.gemm_relu(h, self.w1), self.w2)


class FeedForwardMxfp4:
    """The layer with MXFP4 weights and activations, for inference.

    The weights are stored in-features x out-features, so their columns are
    quantised (``transpose=True``): blocks of 32 along the dimension that the
    product sums over.  No gradient is recorded: the output of an input that
    requires one is detached from it.
    """

    def __init__(self, layer: FeedForward):
        self.eps = layer.eps
        # Copies, as the packed weights are: training the layer further changes neither.
        self.gamma, self.beta = layer.gamma.detach().clone(), layer.beta.detach().clone()
        self.dim, self.hidden = layer.w1.shape
        self.w1 = g.mxfp4_quantize(layer.w1.detach(), transpose=True)
        self.w2 = g.mxfp4_quantize(layer.w2.detach(), transpose=True)

    def __call__(self, x: torch.Tensor) -> torch.Tensor:
        h, _, _ = g.layer_norm_fwd(x, self.gamma, self.beta, eps=self.eps, stats=False)
        a = g.gemm_mxfp4(*g.mxfp4_quantize(h), *self.w1, relu=True, K=self.dim)
        # Through the residual alone a gradient would be wrong.
        return x.detach() + g.gemm_mxfp4(*g.mxfp4_quantize(a), *self.w2, K=self.hidden)


def train(layer: FeedForward, x: torch.Tensor, target: torch.Tensor, steps: int, lr: float = 0.05) -> list[float]:
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
    args = p.parse_args(argv)
    dev = torch.device("cuda", 0)
    gen = torch.Generator(device=dev).manual_seed(1)
    x = torch.randn((args.rows, args.dim), generator=gen, device=dev).half()
    target = torch.randn((args.rows, args.dim), generator=gen, device=dev).half()
    layer = FeedForward(args.dim, args.hidden, device=dev, four_bit=args.four_bit)
    losses = train(layer, x, target, args.steps)
    served = FeedForwardMxfp4(layer)
    with torch.no_grad():
        want, got = layer(x).float(), served(x).float()
        ms16, ms4 = _time(lambda: layer(x)), _time(lambda: served(x))
    st = g.check()
    if st != g.GEMM_OK:
        raise SystemExit(f"device status {st}: {g.strerror(st)}")
    update = (want - x.float()).square().mean().sqrt()
    print(json.dumps({"rows": args.rows, "dim": args.dim, "hidden": args.hidden, "losses": losses, "ms_trained": ms16,
                      "ms_mxfp4": ms4, "rms_difference_of_update": float((want - got).square().mean().sqrt() / update)}))


if __name__ == "__main__":
    main()
