"""A gated feed-forward block of E experts, put together from the package's
operators: router logits [T, E] send each of T tokens to k experts, expert e
maps a row x to W2_e (silu(g) * u) with (g, u) the halves of W1_e x, and the k
results are added with the router's weights.

    ffn_int8   serving: the two products in 8-bit integers
    ffn        training: BF16 products, differentiable in the rows, the logits
               and both weights

Weights are stacked per expert, W1 [E, 2I, H] (gate rows, then up rows) and
W2 [E, H, I].  Derivatives are of first order: a second one through these
operators raises.
"""
import torch

from . import (Routing, moe_combine, moe_combine_grad, moe_dispatch, moe_ffn_int8, moe_route, moe_route_grad,
               quantize_int8)
from .autograd import gradient, grouped_linear


def quantize_weights(W):
    """Codes and scales of stacked weights [E, N, K] (BF16 or FP32), one scale
    per expert and output channel: (int8 [E, N, K], FP32 [E, N])."""
    E, N, K = W.shape
    q, scale = quantize_int8(W.reshape(E * N, K))
    return q.view(E, N, K), scale.view(E, N)


def ffn_int8(X, logits, W1q, w1_scale, W2q, w2_scale, k, renormalize=True):
    """The block on 8-bit weights (codes and scales as quantize_weights gives
    them): X [T, H] BF16 to [T, H] BF16.  Rows are quantised per token before
    each product; the activation between the products stays in FP32 until
    then (rounded to BF16 first, values near the border of two codes would
    take the other one, which moves the result by 0.75 % of its norm).  The
    experts' outputs are rounded to BF16 before they are added in FP32."""
    return moe_ffn_int8(X, logits, W1q, w1_scale, W2q, w2_scale, k, renormalize=renormalize)


class _Route(torch.autograd.Function):
    @staticmethod
    def forward(ctx, logits, k, renormalize):
        r = moe_route(logits, k, renormalize=renormalize)
        ctx.save_for_backward(logits, r.experts, r.weights)
        ctx.renormalize = renormalize
        ctx.mark_non_differentiable(r.experts, r.group_offsets, r.positions, r.tokens)
        return tuple(r)

    @staticmethod
    def backward(ctx, _experts, dweights, _offsets, _positions, _tokens):
        logits, experts, weights = ctx.saved_tensors
        return gradient(lambda *a: moe_route_grad(*a, renormalize=ctx.renormalize), dweights.contiguous(), logits, experts,
                        weights), None, None


class _Dispatch(torch.autograd.Function):
    @staticmethod
    def forward(ctx, X, positions):
        ctx.save_for_backward(positions)
        return moe_dispatch(X, positions)

    @staticmethod
    def backward(ctx, dout):
        return gradient(moe_combine, dout.contiguous(), *ctx.saved_tensors), None


class _Combine(torch.autograd.Function):
    @staticmethod
    def forward(ctx, rows, positions, weights):
        ctx.save_for_backward(rows, positions, weights)
        return moe_combine(rows, positions, weights)

    @staticmethod
    def backward(ctx, dout):
        drows, dweights = gradient(moe_combine_grad, dout.contiguous(), *ctx.saved_tensors)
        return drows, None, dweights


def route(logits, k, renormalize=True):
    """moe_route, differentiable: a Routing whose weights are differentiable in
    the logits."""
    return Routing(*_Route.apply(logits, k, renormalize))


def dispatch(X, positions):
    """moe_dispatch, differentiable in X."""
    return _Dispatch.apply(X, positions)


def combine(rows, positions, weights):
    """The weighted moe_combine, differentiable in rows and weights."""
    return _Combine.apply(rows, positions, weights)


def ffn(X, logits, W1, W2, k, renormalize=True, deterministic=True):
    """The block in BF16, differentiable in X [T, H], logits [T, E] (FP32), W1
    and W2; the weight gradients as autograd.grouped_linear computes them.  What
    passes from one operator to the next is BF16: gate and up, silu(gate), its
    product with up, and the experts' outputs are rounded once each."""
    r = route(logits, k, renormalize)
    gate, up = grouped_linear(dispatch(X, r.positions), W1, r.group_offsets, deterministic).chunk(2, dim=1)
    h = torch.nn.functional.silu(gate) * up
    return combine(grouped_linear(h, W2, r.group_offsets, deterministic), r.positions, r.weights)
