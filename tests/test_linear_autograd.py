"""The products record nothing for autograd: a call whose result would be
expected to have a history is refused, and the same call without that
expectation is not.  On the host, with a stand-in for the library."""
import pytest
import torch

import lossless_compression_float_amd as uz
from test_linear_streams import E, K, M, N, OFF, T, X, packed, streams  # noqa: F401  (a fixture)

BF = torch.bfloat16


def leaf(*shape, dtype=BF):
    return torch.zeros(*shape, dtype=dtype, requires_grad=True)


CALLS = {
    "x": lambda: uz.linear(leaf(M, K), packed(N, K)),
    "bias": lambda: uz.linear(X, packed(N, K), bias=leaf(N)),
    "residual": lambda: uz.linear(X, packed(N, K), residual=leaf(M, N)),
    "out": lambda: uz.linear(X, packed(N, K), out=leaf(M, N)),
    "x of a computation": lambda: uz.linear(leaf(M, K) * 2, packed(N, K)),
    "grouped x": lambda: uz.grouped_linear(leaf(M, K), OFF, packed(E, N, K)),
    "grouped bias": lambda: uz.grouped_linear(X, OFF, packed(E, N, K), bias=leaf(E, N)),
    "loss": lambda: uz.linear_cross_entropy(leaf(M, K), packed(N, K), T),
}


@pytest.mark.parametrize("name", sorted(CALLS))
def test_a_forward_call_that_would_lose_its_gradient_is_refused(streams, name):  # noqa: F811
    with pytest.raises(ValueError, match="autograd"):
        CALLS[name]()
    assert not streams["lib"].calls
    with torch.no_grad():
        CALLS[name]()
    assert streams["lib"].calls


def test_the_pair_of_calls_makes_an_autograd_function(streams):  # noqa: F811
    class Linear(torch.autograd.Function):
        @staticmethod
        def forward(ctx, x, w):
            ctx.save_for_backward(x)
            ctx.w = w
            return uz.linear(x, w)

        @staticmethod
        def backward(ctx, dy):
            x, = ctx.saved_tensors
            return uz.linear_backward(dy.contiguous(), x, ctx.w, need_weight=False)[0], None

    x = leaf(M, K)
    y = Linear.apply(x, packed(N, K))
    assert y.requires_grad
    y.sum().backward()
    assert x.grad.shape == x.shape and streams["lib"].calls.count("uzip_linear_backward") == 1


def test_gradients_may_be_taken_of_leaves(streams):  # noqa: F811
    """The backward calls return gradients, which have no history: leaves may be given as they are."""
    uz.linear_backward(torch.zeros(M, N, dtype=BF), leaf(M, K), packed(N, K))
    uz.linear_cross_entropy_backward(torch.zeros(M), leaf(M, K), packed(N, K), T, torch.zeros(M))
