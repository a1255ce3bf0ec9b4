"""The training operators as differentiable torch functions: the calls of
exact_inner_product_amd.training with their gradients attached.

    from exact_inner_product_amd import autograd as mag
    users = mag.embedding(table, history).mean(1)
    logprobs, _ = mag.item_logprobs(users, items, targets, scale=1 / temperature, bias=-log_q)
    (-logprobs.mean()).backward()
"""
from __future__ import annotations

from typing import Optional, Tuple

import torch

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
