"""The row operators and the router's in torch's autograd: binding.permute, binding.unpermute,
binding.balance_loss and MoeLayer.route of given logits go through these where a gradient is recorded,
so that a training step needs no wiring by hand.

The gradients are the library's own operators; none has a second derivative (asking for one raises). Imported on first use: binding itself loads torch only
inside its functions.
"""
from __future__ import annotations

import torch
from torch.autograd.function import once_differentiable

from . import binding


def _operand(grad):
    """A gradient as the operators take it: contiguous, on a 16-byte boundary (autograd hands on
    expanded ones and views into other tensors)."""
    grad = grad.contiguous()
    return grad if grad.data_ptr() % 16 == 0 else grad.clone()


class Permute(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, rows, n_rows):
        ctx.save_for_backward(rows)
        return binding.permute(x, rows, n_rows)

    @staticmethod
    @once_differentiable
    def backward(ctx, dxs):
        rows, = ctx.saved_tensors
        return binding.permute_backward(_operand(dxs), rows), None, None


class Unpermute(torch.autograd.Function):
    @staticmethod
    def forward(ctx, ys, rows, w, shared, gate, dtype):
        ctx.save_for_backward(ys, rows, w, shared, gate)
        return binding.unpermute(ys, rows, w, shared, gate, dtype)

    @staticmethod
    @once_differentiable
    def backward(ctx, dy):
        ys, rows, w, shared, gate = ctx.saved_tensors
        # a row that no pair names has the gradient 0; the operator leaves it as it was
        dys, dw, dshared, dgate = binding.unpermute_backward(
            _operand(dy), ys, rows, w, shared, gate, dys=torch.zeros_like(ys))
        return dys, None, dw, dshared, dgate, None


class Route(torch.autograd.Function):
    @staticmethod
    def forward(ctx, logits, layer, ws, want_logits):
        z, ids, w, g = layer.route(None, logits.detach(), None, ws, want_logits)
        ctx.save_for_backward(w, ids, g)
        ctx.experts = layer.num_experts
        ctx.mark_non_differentiable(*(t for t in (z, ids) if t is not None))
        return z, ids, w, g

    @staticmethod
    @once_differentiable
    def backward(ctx, dz, dids, dw, dg):
        w, ids, g = ctx.saved_tensors
        dgate = None if g is None else dg.contiguous()
        return binding.route_backward(dw.contiguous(), w, ids, ctx.experts, dgate, g), None, None, None


class BalanceLoss(torch.autograd.Function):
    @staticmethod
    def forward(ctx, logits, ids, num_experts, mask):
        loss, counts, tokens = binding.balance_loss(logits, ids, num_experts, mask)
        # A copy: the caller may sum counts and tokens over ranks in place, and a collective does that
        # without raising the version counter by which autograd would notice.
        kept = torch.cat((counts, tokens.view(1)))
        ctx.save_for_backward(logits, kept, mask)
        ctx.mark_non_differentiable(counts, tokens)
        return loss, counts, tokens

    @staticmethod
    @once_differentiable
    def backward(ctx, dloss, dcounts, dtokens):
        logits, kept, mask = ctx.saved_tensors
        return binding.balance_loss_backward(dloss.contiguous(), logits, kept[:-1], kept[-1], mask), None, None, None
