"""The training operators as differentiable torch functions: the calls of
exact_inner_product_amd.training and .histories with their gradients attached.

    from exact_inner_product_amd import autograd as mag
    events = mag.dropout(mag.embedding(table, history), 0.1, seed, step)
    states, _ = mag.gated_scan(events, torch.nn.functional.linear(events, weight, bias), lengths=lengths)
    users = mag.pool_normalize(states, lengths=lengths)
    logprobs, _ = mag.item_logprobs(users, items, targets, scale=1 / temperature, bias=-log_q)
    (-logprobs.mean()).backward()

Forward and backward passes can be captured into a graph together, as torch's own: on leaves whose gradients no
eager pass that is still alive accumulates (torch.autograd.grad on leaves of the graph's own does).
"""
from __future__ import annotations

from typing import Optional, Tuple

import torch

from .histories import (GatedScan, Pooled, dropout as _dropout, gated_scan as _scan, gated_scan_backward,
                        pool_normalize as _pool, pool_normalize_backward)
from .training import (ItemLogprobs, embedding_grad, embedding_lookup, item_logprobs as _forward,
                       item_logprobs_backward as _backward)


class _ItemLogprobs(torch.autograd.Function):
    @staticmethod
    def forward(ctx, queries, items, ids, bias, exclude, scale, entropy):
        f = _forward(queries, items, ids, scale=scale, bias=bias, exclude=exclude, entropy=entropy)
        ctx.save_for_backward(queries, items, ids, bias, exclude, f.logsumexp, f.entropy)
        ctx.scale = scale
        return f.logprobs, f.entropy

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, grad_logprobs, grad_entropy):
        queries, items, ids, bias, exclude, lse, entropy = ctx.saved_tensors
        need_q, need_i, need_b = ctx.needs_input_grad[0], ctx.needs_input_grad[1], ctx.needs_input_grad[3]
        f = ItemLogprobs(None, lse, entropy, None, None)
        dq, di, db = _backward(grad_logprobs, queries, items, ids, f, scale=ctx.scale, bias=bias, exclude=exclude,
                               grad_entropy=grad_entropy if entropy is not None else None, need_queries=need_q,
                               need_items=need_i, need_bias=need_b)
        return dq, di, None, db, None, None, None


def item_logprobs(queries: torch.Tensor, items: torch.Tensor, ids: torch.Tensor, *, scale: float = 1.0,
                  bias: Optional[torch.Tensor] = None, exclude: Optional[torch.Tensor] = None,
                  entropy: bool = False) -> Tuple[torch.Tensor, Optional[torch.Tensor]]:
    """training.item_logprobs, differentiable in queries, items and bias: (log probabilities
    float32 [b, g], entropy float32 [b] or None)."""
    return _ItemLogprobs.apply(queries, items, ids, bias, exclude, float(scale), entropy)


class _Embedding(torch.autograd.Function):
    @staticmethod
    def forward(ctx, table, ids, scale):
        ctx.save_for_backward(ids)
        ctx.rows, ctx.scale = table.shape[0], scale
        return embedding_lookup(table, ids, scale)

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, grad):
        (ids,) = ctx.saved_tensors
        return embedding_grad(grad, ids, ctx.rows, ctx.scale), None, None


def embedding(table: torch.Tensor, ids: torch.Tensor, scale: float = 1.0) -> torch.Tensor:
    """training.embedding_lookup, differentiable in the table (a dense gradient)."""
    return _Embedding.apply(table, ids, float(scale))


class _GatedScan(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, forget, gate, initial, offsets, lengths, states, grad):
        f = _scan(x, forget, gate, offsets=offsets, lengths=lengths, initial=initial, states=states, carries=grad)
        ctx.save_for_backward(x, forget, gate, initial, offsets, lengths, f.carries)
        ctx.set_materialize_grads(False)  # a result that nothing uses costs its gradient nothing
        return f.states, f.last

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, grad_states, grad_last):
        if grad_states is None and grad_last is None:
            return (None,) * 8
        x, forget, gate, initial, offsets, lengths, carries = ctx.saved_tensors
        dx, df, dg, di = gated_scan_backward(grad_states, grad_last, x, forget, gate, GatedScan(None, None, carries),
                                             offsets=offsets, lengths=lengths, initial=initial)
        return dx, df, dg, di, None, None, None, None


def gated_scan(x: torch.Tensor, forget: torch.Tensor, gate: Optional[torch.Tensor] = None, *,
               offsets: Optional[torch.Tensor] = None, lengths: Optional[torch.Tensor] = None,
               initial: Optional[torch.Tensor] = None, states: bool = True
               ) -> Tuple[Optional[torch.Tensor], torch.Tensor]:
    """histories.gated_scan, differentiable in x, forget, gate and initial: (states, or None if they are
    not wanted; the last ones, float32 [b, d])."""
    grad = torch.is_grad_enabled() and any(t is not None and t.requires_grad for t in (x, forget, gate, initial))
    return _GatedScan.apply(x, forget, gate, initial, offsets, lengths, bool(states), grad)


class _Dropout(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, residual, p, seed, offset, counter):
        ctx.args = (p, seed, offset)
        # the caller advances the counter before the backward pass, which needs the value that was used
        ctx.save_for_backward(None if counter is None else counter.clone())
        ctx.set_materialize_grads(False)
        return _dropout(x, p, seed, offset, residual=residual, counter=counter)

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, grad):
        if grad is None:
            return (None,) * 6
        (counter,) = ctx.saved_tensors
        dx = _dropout(grad, *ctx.args, counter=counter) if ctx.needs_input_grad[0] else None
        return dx, grad if ctx.needs_input_grad[1] else None, None, None, None, None


def dropout(x: torch.Tensor, p: float, seed: int, offset: int = 0, *, residual: Optional[torch.Tensor] = None,
            counter: Optional[torch.Tensor] = None) -> torch.Tensor:
    """histories.dropout, differentiable in x and residual."""
    return _Dropout.apply(x, residual, p, seed, offset, counter)


class _Pool(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, offsets, lengths, normalize):
        f = _pool(x, offsets=offsets, lengths=lengths, normalize=normalize)
        ctx.save_for_backward(offsets, lengths, f.mean, f.norm)
        ctx.shape, ctx.normalize = x.shape, normalize
        return f.vectors

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, grad):
        offsets, lengths, mean, norm = ctx.saved_tensors
        f = Pooled(grad, mean, norm, ctx.normalize)  # (the vectors give their type and shape only)
        return pool_normalize_backward(grad, ctx.shape, f, offsets=offsets, lengths=lengths), None, None, None


def pool_normalize(x: torch.Tensor, *, offsets: Optional[torch.Tensor] = None,
                   lengths: Optional[torch.Tensor] = None, normalize: bool = True) -> torch.Tensor:
    """histories.pool_normalize's vectors, differentiable in x."""
    return _Pool.apply(x, offsets, lengths, bool(normalize))
