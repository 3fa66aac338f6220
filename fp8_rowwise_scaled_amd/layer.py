"""Python entry points of the layer operators (include/fp8gg_layer.h).

Arguments go to the compiled module _layer_binding, which checks the tensors, allocates
the outputs and workspaces that are not given on the inputs' device, and makes the
library's call on the current stream.  There is no fallback: without the built library
and module these functions raise.
"""
from __future__ import annotations

import importlib
from typing import NamedTuple, Optional

import torch

from . import _lib

_SCORES = {"softmax": _lib.SCORE_SOFTMAX, "sigmoid": _lib.SCORE_SIGMOID}
_module = None


def _binding():
    """The compiled module; raises if it has not been built."""
    global _module
    if _module is None:
        _lib.load()
        try:
            _module = importlib.import_module("._layer_binding", __package__)
        except ImportError as e:
            raise RuntimeError("_layer_binding.so is missing or does not load: build it with `python -m "
                               f"fp8_rowwise_scaled_amd.build` (there is no fallback implementation): {e}") from e
    return _module


class RmsNorm(NamedTuple):
    XQ: torch.Tensor
    x_scale: torch.Tensor
    residual: Optional[torch.Tensor]
    Y: Optional[torch.Tensor]
    rstd: Optional[torch.Tensor]


class Route(NamedTuple):
    weights: torch.Tensor
    ids: torch.Tensor
    M_sizes: Optional[torch.Tensor]
    dst_row: Optional[torch.Tensor]


class SiluMul(NamedTuple):
    AQ: torch.Tensor
    a_scale: torch.Tensor
    HQ: Optional[torch.Tensor]
    h_scale: Optional[torch.Tensor]


def _score(score: str) -> int:
    code = _SCORES.get(score)
    if code is None:
        raise ValueError(f"score must be 'softmax' or 'sigmoid', got {score!r}")
    return code


def f8f8bf16_rmsnorm_quantize(X, weight, eps=1e-6, residual=None, block=0, want_y=False, want_rstd=False, XQ=None,
                              x_scale=None, residual_out=None, Y=None, rstd=None) -> RmsNorm:
    """Root-mean-square norm of X + residual with an fp8 output: X [rows, K] bf16,
    weight [K] bf16 or float32, residual [rows, K] bf16 or None; block 0 gives one
    scale per row, 128 one per row and 128 columns.  Returns RmsNorm(XQ uint8 codes,
    x_scale, residual = bf16(X + residual) or None, Y bf16 if wanted or given, rstd if
    wanted or given).  residual_out may be residual itself (see include/fp8gg_layer.h)."""
    return RmsNorm._make(_binding().rmsnorm_quantize(X, weight, eps, residual, block, want_y, want_rstd, XQ, x_scale,
                                                     residual_out, Y, rstd))


def f8f8bf16_rmsnorm_backward(dY, H, weight, rstd, dresidual=None, dX=None, dweight=None, workspace=None):
    """Gradient of the norm: dY and H (the forward's X + residual) [rows, K] bf16, rstd
    [rows] of the forward pass, dresidual [rows, K] bf16 the gradient that reaches the
    residual output, or None.  Returns (dX bf16, the gradient of X and residual alike,
    dweight float32 [K]).  dX may be dY or dresidual itself."""
    return _binding().rmsnorm_backward(dY, H, weight, rstd, dresidual, dX, dweight, workspace)


def f8f8bf16_route(logits, k, bias=None, score="softmax", n_group=1, topk_group=1, group_top=1, renormalize=True,
                   scale=1.0, plan=True, weights=None, ids=None, M_sizes=None, dst_row=None, workspace=None) -> Route:
    """Routes tokens to experts: logits [T, E] float32 or bf16, bias [E] float32 added to
    the scores for the choice only, n_group groups of neighbouring experts of which the
    topk_group best (by the sum of their group_top highest keys) stay.  Returns
    Route(weights float32 [T, k], ids int32 [T, k], M_sizes int64 [E], dst_row int32
    [T, k]); the last two are None with plan=False (see include/fp8gg_layer.h)."""
    return Route._make(_binding().route(logits, k, bias, _score(score), n_group, topk_group, group_top, renormalize, scale,
                                        plan, weights, ids, M_sizes, dst_row, workspace))


def f8f8bf16_route_backward(logits, ids, dweights, score="softmax", renormalize=True, scale=1.0, dlogits=None):
    """Gradient of the routing weights with respect to the logits, the choice held fixed:
    ids int32 [T, k] and dweights float32 [T, k]; returns dlogits [T, E] of logits' type."""
    return _binding().route_backward(logits, ids, dweights, _score(score), renormalize, scale, dlogits)


def f8f8bf16_moe_dispatch(XQ, x_scale, dst_row, rows=None, XQs=None, xs_out=None):
    """Copies codes XQ [T, K] and scales x_scale ([T] or [T, K / 128]) to the experts'
    order: row dst_row[t, j] of the outputs is row t, for every j.  Returns (XQs
    [rows, K], xs_out), rows = T * k unless given; entries of dst_row outside
    [0, rows) are left out, rows that no entry names are not written."""
    return _binding().moe_dispatch(XQ, x_scale, dst_row, rows, XQs, xs_out)


def f8f8bf16_moe_combine(Y, dst_row, weights=None, addend=None, out=None):
    """out[t] = sum_j weights[t, j] * Y[dst_row[t, j]] + addend[t]: Y [R, N] bf16, dst_row
    int32 [T, k], weights float32 [T, k] (None: ones), addend [T, N] bf16 or None.
    Returns out [T, N] bf16, which may be addend itself."""
    return _binding().moe_combine(Y, dst_row, weights, addend, out)


def f8f8bf16_moe_combine_backward(dout, dst_row, weights=None, Y=None, rows=None, dY=None, dweights=None):
    """Gradients of combine: dout [T, N] bf16, Y [R, N] the forward's rows (None: no
    gradient of the weights, and rows gives R, T * k by default).  Returns (dY [R, N]
    bf16, dweights float32 [T, k] or None); rows of dY that no entry of dst_row names are
    not written, and two entries must not name the same row.  With weights and Y None it is
    a dispatch of bf16 rows."""
    return _binding().moe_combine_backward(dout, dst_row, weights, Y, rows, dY, dweights)


def f8f8bf16_silu_mul_quantize(H, block=0, checkpoint=False, AQ=None, a_scale=None, HQ=None, h_scale=None) -> SiluMul:
    """silu(gate) * up of H = [gate | up] [rows, 2 I] bf16 with an fp8 output (block as in
    rmsnorm_quantize) and, with checkpoint=True (or HQ and h_scale given), the 8-bit
    checkpoint of H that silu_mul_backward reads.  Returns SiluMul(AQ [rows, I], a_scale,
    HQ [rows, 2 I] or None, h_scale [rows, 2, ceil(I / 128)] or None)."""
    return SiluMul._make(_binding().silu_mul_quantize(H, block, checkpoint, AQ, a_scale, HQ, h_scale))


def f8f8bf16_silu_mul_backward(dA, HQ, h_scale, dH=None):
    """Gradient of silu(gate) * up from the 8-bit checkpoint: dA [rows, I] bf16; returns
    dH [rows, 2 I] bf16."""
    return _binding().silu_mul_backward(dA, HQ, h_scale, dH)


def f8f8bf16_k_offsets_capacity(R: int, G: int) -> int:
    """Columns that quantize_k_offsets needs for R rows in G groups."""
    return _lib.load().f8f8bf16_k_offsets_capacity(R, G)


def f8f8bf16_quantize_k_offsets(X, M_sizes, x_scale=None, XT=None, t_scale=None, k_offsets=None, workspace=None):
    """The weight gradient's operand from rows in expert order: X [R, K] bf16, or fp8
    codes with x_scale ([R] or [R, K / 128]); M_sizes int64 [G].  Returns (XT uint8
    [K, capacity], t_scale float32 [G, K], k_offsets int32 [G]), an operand of
    f8f8bf16_rowwise_grouped_k_offsets with its scales and offsets."""
    return _binding().quantize_k_offsets(X, M_sizes, x_scale, XT, t_scale, k_offsets, workspace)
