"""Python entry points of the training operators (include/fp8gg_train.h).

As for the layer operators, arguments go to the compiled module _layer_binding, which
checks the tensors, allocates the outputs and workspaces that are not given on the inputs'
device, and makes the library's call on the current stream.
"""
from __future__ import annotations

from typing import NamedTuple, Optional

import torch

from .layer import _binding

_DTYPES = (torch.float32, torch.bfloat16)


class WeightBlocks(NamedTuple):
    WQ: torch.Tensor
    w_scale: torch.Tensor
    WQt: Optional[torch.Tensor]
    wt_scale: Optional[torch.Tensor]


def bf16_grouped_stacked(X, W, M_sizes, Y=None):
    """Y[m] = X[m] @ W[g].T for the rows m of each group g: X [total_M, K] and W [G, N, K]
    bf16, M_sizes int64 [G].  Returns Y [total_M, N] bf16; rows past the groups' end are not
    written."""
    return _binding().grouped_product(X, W, M_sizes, Y)


def bf16_grouped_stacked_dgrad(dY, W, M_sizes, dX=None):
    """The gradient of bf16_grouped_stacked's X: dX[m] = dY[m] @ W[g], dY [total_M, N] and
    W [G, N, K] bf16.  Returns dX [total_M, K] bf16."""
    return _binding().grouped_dgrad(dY, W, M_sizes, dX)


def bf16_grouped_stacked_wgrad(dY, X, M_sizes, dtype=torch.float32, dW=None, accumulate=False, workspace=None):
    """The gradient of bf16_grouped_stacked's W: dW[g] = dY[rows of g].T @ X[rows of g],
    dY [total_M, N] and X [total_M, K] bf16.  Returns dW [G, N, K] of the dtype (float32 or
    bfloat16; a given dW's own); with accumulate (float32 only, dW given) it is added to what
    dW holds."""
    if dtype not in _DTYPES:
        raise ValueError(f"dtype must be torch.float32 or torch.bfloat16, got {dtype}")
    return _binding().grouped_wgrad(dY, X, M_sizes, dtype is torch.float32, dW, accumulate, workspace)


def f8f8bf16_quantize_groupwise(X, XQ=None, x_scale=None):
    """Rows as an operand of the block-scaled products: X [rows, K] bf16, K a multiple of
    128.  Returns (XQ uint8 codes [rows, K], x_scale float32 [rows, K / 128])."""
    return _binding().quantize_groupwise(X, XQ, x_scale)


def f8f8bf16_quantize_groupwise_weight(W, transposed=False, WQ=None, w_scale=None, WQt=None, wt_scale=None) -> WeightBlocks:
    """Weights as operands of the block-scaled products: W [G, N, K] (or [N, K]) bf16 or
    float32, N and K multiples of 128.  Returns WeightBlocks(WQ uint8 codes of W's shape,
    w_scale float32 [G, N / 128, K / 128], and with transposed=True (or WQt and wt_scale
    given) WQt [G, K, N] and wt_scale [G, K / 128, N / 128] of the same codes, else None)."""
    return WeightBlocks._make(_binding().quantize_weight(W, transposed, WQ, w_scale, WQt, wt_scale))


def f8f8bf16_grad_square_sum(grads, square_sum=None, workspace=None):
    """The sum of all values' squares, float64 [1], of a list of float32 or bf16 tensors on
    one device."""
    return _binding().grad_square_sum(grads, square_sum, workspace)


def f8f8bf16_grad_clip(grads, max_norm, eps=1e-6, square_sum=None, outs=None, norm=None, workspace=None):
    """Scales a list of float32 or bf16 gradients by min(1, max_norm / (norm + eps)), in
    place or into the tensors of outs (of the same shapes, types and strides).  An infinite
    max_norm leaves every value as it is, whatever the norm.  norm is the
    square root of square_sum (float64 [1], as grad_square_sum gives it) or, if that is None,
    of the gradients' own.  Returns norm, float32 [1], on the device."""
    return _binding().grad_clip(grads, max_norm, eps, square_sum, outs, norm, workspace)
