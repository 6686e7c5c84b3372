"""Refusals of the feed-forward layer's functions that need no GPU."""
from __future__ import annotations

import types

import pytest
import torch

from dense_fp16_gemm_05_gb300 import build as gbuild


@pytest.fixture(scope="module")
def ag():
    gbuild.build()
    from dense_fp16_gemm_05_gb300 import autograd, gemm_f16
    gemm_f16.lib()
    return autograd


@pytest.mark.parametrize("a,b", [((4, 40), (48, 8)), ((4, 33), (64, 8)), ((4, 64), (63, 8)), ((4, 64), (96, 8))])
def test_four_bit_linear_refuses_inner_sizes_that_differ(ag, a, b):
    # also those that fill the same number of blocks of 32
    with pytest.raises(ValueError, match="inner sizes differ"):
        ag.linear_mxfp4(torch.zeros(a, dtype=torch.float16), torch.zeros(b, dtype=torch.float16))


H, BF, F = torch.float16, torch.bfloat16, torch.float32


# dA is a product with B's values, dB one with A's, both over rows of K
@pytest.mark.parametrize("K,ta,tb,which", [(64, BF, BF, "A"), (64, F, F, "B"), (64, H, BF, "A"), (64, BF, H, "B"),
                                           (64, H, F, "AB"), (36, H, H, "A"), (36, H, H, "B"), (4, H, H, "AB")])
def test_four_bit_linear_refuses_at_the_call_what_its_gradients_do_not_take(ag, K, ta, tb, which):
    A = torch.zeros((4, K), dtype=ta, requires_grad="A" in which)
    B = torch.zeros((K, 8), dtype=tb, requires_grad="B" in which)
    with pytest.raises(ValueError, match="for the gradients"):
        ag.linear_mxfp4(A, B)


@pytest.fixture
def ff(ag, monkeypatch):
    """The example with the operators' results replaced by zeros of their shapes."""
    from dense_fp16_gemm_05_gb300 import feed_forward
    shapes = {"mxfp4_quantize": lambda x, transpose=False: (x.detach().t() if transpose else x.detach(), None),
              "gemm_mxfp4": lambda a, sa, w, sw, **kw: torch.zeros((a.shape[0], w.shape[0]), dtype=H),
              "layer_norm_fwd": lambda x, gamma, beta, eps, stats: (x.detach() * gamma + beta, None, None)}
    monkeypatch.setattr(feed_forward, "g", types.SimpleNamespace(**shapes))
    return feed_forward


def test_served_layer_gives_no_gradient(ff):
    # the residual's gradient alone would be a wrong one
    served = ff.FeedForwardMxfp4(ff.FeedForward(64, 128, device="cpu"))
    x = torch.ones((4, 64), dtype=H, requires_grad=True)
    y = served(x)
    assert not y.requires_grad and torch.equal(y, x.detach()) and x.grad is None


def test_served_layer_is_the_layer_as_it_was_converted(ff):
    layer = ff.FeedForward(64, 128, device="cpu")
    served = ff.FeedForwardMxfp4(layer)
    with torch.no_grad():
        layer.gamma += 1.0
        layer.beta -= 1.0
    assert (served.gamma == 1.0).all() and (served.beta == 0.0).all()
