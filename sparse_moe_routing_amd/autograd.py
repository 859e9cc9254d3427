"""The row operators in torch's autograd: binding.permute and binding.unpermute go through these
where a gradient is recorded, so that a training step needs no wiring by hand.

Both gradients are the library's own operators and exact transposes of the forward pass; neither has
a second derivative (asking for one raises). Imported on first use: binding itself loads torch only
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
