"""torch.autograd wrapper around the library's kernels (training use).

The TileLang-MUSA lesson (7yue.com, section 6, "wrapping a TileLang kernel for
PyTorch") wraps its GEMM kernel in a ``torch.autograd.Function`` whose forward
calls the kernel and whose backward returns ``dA = dC @ B.T`` and
``dB = A.T @ dC``.  Here every step runs in this library's sm_103a kernels:

* forward   C = R(A @ B)                         gemm_f16_tx (NN)
* ReLU      dZ = dC where C > 0, else +0         gemm_f16_relu_backward (only with ReLU)
* dA        dZ @ B^T   (B stored (K,N))          gemm_f16_tx with transb = 1 (NT)
* dB        A^T @ dZ   (A stored (M,K))          gemm_f16_tx with transa = 1 (TN)

and, for the block around them, layer norm (layer_norm_fwd, layer_norm_bwd), RMS
norm with the residual's addition (rms_norm_fwd, rms_norm_bwd), dropout whose mask
is never stored, and the product of MXFP4-quantised operands with gradients passed
straight through the quantisation.

The GEMMs' operands and gradients are float16 (the kernels accumulate in fp32).  No step
falls back to torch arithmetic; a missing library raises LibraryNotBuilt.
"""
from __future__ import annotations

import torch

from . import gemm_f16 as _g


class GemmF16Function(torch.autograd.Function):
    """C = ReLU(A @ B) (relu=True) or A @ B, with the backward pair above."""

    @staticmethod
    def forward(ctx, A: torch.Tensor, B: torch.Tensor, relu: bool = True):
        A = A.contiguous()
        B = B.contiguous()
        C = _g.gemm_f16_t(A, B, relu=relu)
        ctx.relu = bool(relu)
        ctx.save_for_backward(A, B, C if relu else None)
        return C

    @staticmethod
    def backward(ctx, dC: torch.Tensor):
        A, B, C = ctx.saved_tensors
        dC = dC.contiguous()
        if dC.dtype != torch.float16:
            dC = dC.half()
        dZ = _g.relu_backward(dC, C) if ctx.relu else dC
        dA = dB = None
        if ctx.needs_input_grad[0]:
            dA = _g.gemm_f16_t(dZ, B, transb=True, relu=False)     # (M,N) @ (N,K)
        if ctx.needs_input_grad[1]:
            dB = _g.gemm_f16_t(A, dZ, transa=True, relu=False)     # (K,M) @ (M,N)
        return dA, dB, None


class LinearMxfp4Function(torch.autograd.Function):
    """R(q(A) @ q(B)) with q the MXFP4 quantisation along the summed dimension.

    The gradients are those of the product of the quantised values, passed
    straight through the quantisation (whose own derivative is zero almost
    everywhere): dA = dZ @ q(B)^T, dB = q(A)^T @ dZ, in the fp16 GEMMs.
    """

    @staticmethod
    def forward(ctx, A: torch.Tensor, B: torch.Tensor, relu: bool):
        A, B = A.contiguous(), B.contiguous()
        need_a, need_b = ctx.needs_input_grad[0], ctx.needs_input_grad[1]
        qa = _g.mxfp4_quantize(A, values=need_b)
        qb = _g.mxfp4_quantize(B, transpose=True, values=need_a)
        C = _g.gemm_mxfp4(qa[0], qa[1], qb[0], qb[1], relu=relu, K=A.shape[1])
        ctx.relu = relu
        # q(A) (M,K) and q(B)^T (N,K), as fp16 values.
        ctx.save_for_backward(qa[2] if need_b else None, qb[2] if need_a else None, C if relu else None)
        return C

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dC: torch.Tensor):
        Av, Bv, C = ctx.saved_tensors
        dC = dC.contiguous()
        if dC.dtype != torch.float16:
            dC = dC.half()
        dZ = _g.relu_backward(dC, C) if ctx.relu else dC
        dA = dB = None
        if ctx.needs_input_grad[0]:
            dA = _g.gemm_f16_t(dZ, Bv, relu=False)                  # (M,N) @ (N,K)
        if ctx.needs_input_grad[1]:
            dB = _g.gemm_f16_t(Av, dZ, transa=True, relu=False)     # (K,M) @ (M,N)
        return dA, dB, None


class LayerNormFunction(torch.autograd.Function):
    """Layer norm over the last dimension; its backward is layer_norm_bwd."""

    @staticmethod
    def forward(ctx, x: torch.Tensor, gamma: torch.Tensor | None, beta: torch.Tensor | None, eps: float):
        x = x.contiguous()
        y, mean, rstd = _g.layer_norm_fwd(x, gamma, beta, eps=eps)
        ctx.save_for_backward(x, gamma, mean, rstd)
        ctx.wtype = beta.dtype if gamma is None and beta is not None else None
        return y

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dy: torch.Tensor):
        x, gamma, mean, rstd = ctx.saved_tensors
        dy = dy.contiguous()
        if dy.dtype != x.dtype:
            dy = dy.to(x.dtype)
        need_g, need_b = ctx.needs_input_grad[1], ctx.needs_input_grad[2]
        dx, dgamma, dbeta = _g.layer_norm_bwd(dy, x, mean, rstd, gamma, weights=need_g or need_b, wtype=ctx.wtype)
        return (dx if ctx.needs_input_grad[0] else None, dgamma if need_g else None, dbeta if need_b else None, None)


class RmsNormFunction(torch.autograd.Function):
    """(Y, H): RMS norm of H = x + residual over the last dimension; Y alone without a residual."""

    @staticmethod
    def forward(ctx, x: torch.Tensor, gamma: torch.Tensor | None, residual: torch.Tensor | None, eps: float):
        x = x.contiguous()
        y, h, rstd = _g.rms_norm_fwd(x, gamma, None if residual is None else residual.contiguous(), eps=eps)
        ctx.save_for_backward(h, gamma, rstd)
        ctx.set_materialize_grads(False)
        return y if residual is None else (y, h)

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dy: torch.Tensor | None, dh: torch.Tensor | None = None):
        h, gamma, rstd = ctx.saved_tensors
        need_x, need_g, need_r, _ = ctx.needs_input_grad
        if dh is not None:
            dh = dh.contiguous().to(h.dtype)
        if dy is None:   # only the stream was used
            return (dh if need_x else None, torch.zeros_like(gamma) if need_g else None, dh if need_r else None, None)
        dx, dgamma = _g.rms_norm_bwd(dy.contiguous().to(h.dtype), h, rstd, gamma, dH=dh, weights=need_g)
        return dx if need_x else None, dgamma, dx if need_r else None, None


class DropoutFunction(torch.autograd.Function):
    """residual + x / (1 - p) where an element is kept; the backward pass makes the mask again."""

    @staticmethod
    def forward(ctx, x: torch.Tensor, p: float, seed: int, offset, residual: torch.Tensor | None):
        y = _g.dropout(x.contiguous(), p, seed, offset, residual=None if residual is None else residual.contiguous())
        ctx.p, ctx.seed = p, seed
        # Saved, so that a change of it in between is an error and not another mask.
        ctx.save_for_backward(offset if isinstance(offset, torch.Tensor) else None)
        ctx.offset = None if isinstance(offset, torch.Tensor) else offset
        return y

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dy: torch.Tensor):
        (offset,) = ctx.saved_tensors
        dx = None
        if ctx.needs_input_grad[0]:
            dx = _g.dropout(dy.contiguous(), ctx.p, ctx.seed, ctx.offset if offset is None else offset)
        return dx, None, None, None, dy if ctx.needs_input_grad[4] else None


def linear_mxfp4(A: torch.Tensor, B: torch.Tensor, relu: bool = False) -> torch.Tensor:
    """C = A @ B or ReLU(A @ B) with both operands quantised to MXFP4, for training with 4-bit products.

    A (M,K) and B (K,N): float16 CUDA tensors, K and N multiples of 8 (the
    gradients' GEMMs); where no gradient is recorded any K and the quantiser's
    other types serve too.  Straight-through gradients, see LinearMxfp4Function.
    """
    if A.dim() == 2 and B.dim() == 2 and A.shape[1] != B.shape[0]:
        # Their packed forms would not tell: K is rounded up to whole blocks there.
        raise ValueError(f"inner sizes differ: A {tuple(A.shape)}, B {tuple(B.shape)}")
    if torch.is_grad_enabled() and (A.requires_grad or B.requires_grad):
        # Here and not in the backward pass, whose fp16 GEMMs would refuse: either
        # gradient is a product with the other operand's values.
        for t, other, name in ((A, B, "A"), (B, A, "B")):
            if other.requires_grad and t.dtype != torch.float16:
                raise ValueError(f"{name} must be float16 for the gradients, got {t.dtype}")
        if A.dim() == 2 and A.shape[1] % 8:
            raise ValueError(f"K must be a multiple of 8 for the gradients, got {A.shape[1]}")
    return LinearMxfp4Function.apply(A, B, bool(relu))


def layer_norm(x: torch.Tensor, gamma: torch.Tensor | None = None, beta: torch.Tensor | None = None,
               eps: float = 1e-5) -> torch.Tensor:
    """Differentiable layer norm over x's last dimension on CUDA tensors.

    As with any torch function, capture a training step's backward pass only
    with its forward pass, after warm-up on the capture stream and with no
    eager graph of the same leaves alive.
    """
    return LayerNormFunction.apply(x, gamma, beta, eps)


def rms_norm(x: torch.Tensor, gamma: torch.Tensor | None = None, eps: float = 1e-6,
             residual: torch.Tensor | None = None):
    """Differentiable RMS norm over x's last dimension on CUDA tensors.

    With ``residual`` (x's shape and type) it returns (Y, H): H = x + residual, the
    residual stream, and Y its norm; the gradients that reach H past the norm are
    added in the backward kernel.  Without one it returns Y, the norm of x.
    Capturing a backward pass: as for layer_norm.
    """
    return RmsNormFunction.apply(x, gamma, residual, eps)


def dropout(x: torch.Tensor, p: float, seed: int, offset: int | torch.Tensor = 0,
            residual: torch.Tensor | None = None) -> torch.Tensor:
    """Differentiable residual + x / (1 - p) where an element is kept, residual (0 without one) where not.

    The mask is a function of ``seed``, ``offset`` and the element's place (see
    gemm_f16.dropout) and is not stored.  ``offset`` may be an int64 CUDA tensor of
    one element, for captured steps that advance it; it must not change between the
    forward and the backward pass.
    """
    return DropoutFunction.apply(x, p, seed, offset, residual)


def gemm_relu(A: torch.Tensor, B: torch.Tensor) -> torch.Tensor:
    """Differentiable C = ReLU(A @ B) on fp16 CUDA tensors."""
    return GemmF16Function.apply(A, B, True)


def gemm(A: torch.Tensor, B: torch.Tensor) -> torch.Tensor:
    """Differentiable C = A @ B on fp16 CUDA tensors (the lesson's TLGemm)."""
    return GemmF16Function.apply(A, B, False)
