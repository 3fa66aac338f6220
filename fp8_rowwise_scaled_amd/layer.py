"""Python entry points of the layer operators (include/fp8gg_layer.h): argument
marshalling only, as in ops.py.  Outputs and workspaces that are not given are
allocated on the inputs' device; the work goes to the current stream.
"""
from __future__ import annotations

from typing import NamedTuple, Optional

import torch

from . import _lib
from .ops import _bytes, _check, _refuse, _stream

_SCORES = {"softmax": _lib.SCORE_SOFTMAX, "sigmoid": _lib.SCORE_SIGMOID}
_FLOATS = {torch.bfloat16: _lib.DTYPE_BF16, torch.float32: _lib.DTYPE_F32}


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


def _float_type(t: torch.Tensor, name: str) -> int:
    code = _FLOATS.get(t.dtype)
    if code is None:
        raise ValueError(f"{name} must be bfloat16 or float32, got {t.dtype}")
    return code


def _same_device(first: torch.Tensor, *others) -> None:
    for t in others:
        if t is not None and t.device != first.device:
            raise ValueError(f"all tensors must be on one device, got {first.device} and {t.device}")


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else t.data_ptr()


def _matrix(t: torch.Tensor, name: str, dtype, shape: str) -> tuple:
    """Rows and columns of a 2-D contiguous GPU tensor."""
    if t.dim() != 2:
        raise ValueError(f"{name} must be {shape}")
    if t.dtype != dtype or not t.is_cuda or not t.is_contiguous():
        _refuse(t, name, dtype, tuple(t.shape))
    return t.shape


def _given(t: Optional[torch.Tensor], name: str, dtype, shape: tuple, dev: torch.device) -> torch.Tensor:
    """The caller's output, checked, or a new one."""
    if t is None:
        return torch.empty(shape, dtype=dtype, device=dev)
    if dtype == torch.uint8:
        t = _bytes(t, name)
    _check(t, name, dtype, shape)
    if t.device != dev:
        raise ValueError(f"{name} must be on {dev}")
    return t


def _workspace(t: Optional[torch.Tensor], need: int, dev: torch.device) -> tuple:
    """(pointer, bytes) of the caller's workspace or of a new one.  A new one may be
    released when the call returns: the allocator hands it out again in stream order."""
    if t is None:
        if need == 0:
            return None, 0, None
        t = torch.empty((need,), dtype=torch.uint8, device=dev)
    elif not t.is_cuda or not t.is_contiguous() or t.device != dev:
        raise ValueError(f"workspace must be contiguous and on {dev}")
    return t.data_ptr(), t.numel() * t.element_size(), t


def _block_cols(block: int, K: int) -> int:
    if block not in (0, 128):
        raise ValueError(f"block must be 0 (one scale per row) or 128, got {block}")
    if block and K % 128:
        raise ValueError(f"block scaling needs a multiple of 128 columns, got {K}")
    return K // 128 if block else 0


def f8f8bf16_rmsnorm_quantize(X, weight, eps=1e-6, residual=None, block=0, want_y=False, want_rstd=False, XQ=None,
                              x_scale=None, residual_out=None, Y=None, rstd=None) -> RmsNorm:
    """Root-mean-square norm of X + residual with an fp8 output: X [rows, K] bf16,
    weight [K] bf16 or float32, residual [rows, K] bf16 or None; block 0 gives one
    scale per row, 128 one per row and 128 columns.  Returns RmsNorm(XQ uint8 codes,
    x_scale, residual = bf16(X + residual) or None, Y bf16 if wanted or given, rstd if
    wanted or given).  residual_out may be residual itself (see include/fp8gg_layer.h)."""
    rows, K = _matrix(X, "X", torch.bfloat16, "[rows, K]")
    dev = X.device
    wt = _float_type(weight, "weight")
    _check(weight, "weight", weight.dtype, (K,))
    _same_device(X, weight, residual)
    cols = _block_cols(block, K)
    XQ = _given(XQ, "XQ", torch.uint8, (rows, K), dev)
    x_scale = _given(x_scale, "x_scale", torch.float32, (rows, cols) if cols else (rows,), dev)
    if residual is not None:
        _check(residual, "residual", torch.bfloat16, (rows, K))
        residual_out = _given(residual_out, "residual_out", torch.bfloat16, (rows, K), dev)
    elif residual_out is not None:
        raise ValueError("residual_out is given without a residual")
    if want_y or Y is not None:
        Y = _given(Y, "Y", torch.bfloat16, (rows, K), dev)
    if want_rstd or rstd is not None:
        rstd = _given(rstd, "rstd", torch.float32, (rows,), dev)
    st = _lib.load().f8f8bf16_rmsnorm_quantize(
        X.data_ptr(), _ptr(residual), weight.data_ptr(), wt, eps, block, XQ.data_ptr(), x_scale.data_ptr(), _ptr(Y),
        _ptr(residual_out), _ptr(rstd), rows, K, _stream(dev))
    if st:
        _lib.layer_check(st, "f8f8bf16_rmsnorm_quantize")
    return RmsNorm(XQ, x_scale, residual_out, Y, rstd)


def f8f8bf16_rmsnorm_backward(dY, H, weight, rstd, dresidual=None, dX=None, dweight=None, workspace=None):
    """Gradient of the norm: dY and H (the forward's X + residual) [rows, K] bf16, rstd
    [rows] of the forward pass, dresidual [rows, K] bf16 the gradient that reaches the
    residual output, or None.  Returns (dX bf16, the gradient of X and residual alike,
    dweight float32 [K]).  dX may be dY or dresidual itself."""
    rows, K = _matrix(dY, "dY", torch.bfloat16, "[rows, K]")
    dev = dY.device
    _check(H, "H", torch.bfloat16, (rows, K))
    wt = _float_type(weight, "weight")
    _check(weight, "weight", weight.dtype, (K,))
    _check(rstd, "rstd", torch.float32, (rows,))
    if dresidual is not None:
        _check(dresidual, "dresidual", torch.bfloat16, (rows, K))
    _same_device(dY, H, weight, rstd, dresidual)
    dX = _given(dX, "dX", torch.bfloat16, (rows, K), dev)
    dweight = _given(dweight, "dweight", torch.float32, (K,), dev)
    lib = _lib.load()
    ws, size, _hold = _workspace(workspace, lib.f8f8bf16_rmsnorm_backward_workspace(rows, K), dev)
    st = lib.f8f8bf16_rmsnorm_backward(dY.data_ptr(), H.data_ptr(), weight.data_ptr(), wt, rstd.data_ptr(),
                                       _ptr(dresidual), dX.data_ptr(), dweight.data_ptr(), ws, size, rows, K, _stream(dev))
    if st:
        _lib.layer_check(st, "f8f8bf16_rmsnorm_backward")
    return dX, dweight


def _score(score: str) -> int:
    code = _SCORES.get(score)
    if code is None:
        raise ValueError(f"score must be 'softmax' or 'sigmoid', got {score!r}")
    return code


def _logits(logits: torch.Tensor) -> tuple:
    code = _float_type(logits, "logits")
    return (code, *_matrix(logits, "logits", logits.dtype, "[T, E]"))


def f8f8bf16_route(logits, k, bias=None, score="softmax", n_group=1, topk_group=1, group_top=1, renormalize=True,
                   scale=1.0, plan=True, weights=None, ids=None, M_sizes=None, dst_row=None, workspace=None) -> Route:
    """Routes tokens to experts: logits [T, E] float32 or bf16, bias [E] float32 added to
    the scores for the choice only, n_group groups of neighbouring experts of which the
    topk_group best (by the sum of their group_top highest keys) stay.  Returns
    Route(weights float32 [T, k], ids int32 [T, k], M_sizes int64 [E], dst_row int32
    [T, k]); the last two are None with plan=False (see include/fp8gg_layer.h)."""
    dt, T, E = _logits(logits)
    dev = logits.device
    if bias is not None:
        _check(bias, "bias", torch.float32, (E,))
        _same_device(logits, bias)
    weights = _given(weights, "weights", torch.float32, (T, k), dev)
    ids = _given(ids, "ids", torch.int32, (T, k), dev)
    lib = _lib.load()
    ws, size, _hold = None, 0, None
    if plan:
        M_sizes = _given(M_sizes, "M_sizes", torch.int64, (E,), dev)
        dst_row = _given(dst_row, "dst_row", torch.int32, (T, k), dev)
        ws, size, _hold = _workspace(workspace, lib.f8f8bf16_route_workspace(T, E, k), dev)
    elif M_sizes is not None or dst_row is not None:
        raise ValueError("M_sizes and dst_row are outputs of the plan, which plan=False leaves out")
    st = lib.f8f8bf16_route(logits.data_ptr(), dt, _ptr(bias), _score(score), n_group, topk_group, group_top,
                            1 if renormalize else 0, scale, weights.data_ptr(), ids.data_ptr(), _ptr(M_sizes),
                            _ptr(dst_row), ws, size, T, E, k, _stream(dev))
    if st:
        _lib.layer_check(st, "f8f8bf16_route")
    return Route(weights, ids, M_sizes, dst_row)


def f8f8bf16_route_backward(logits, ids, dweights, score="softmax", renormalize=True, scale=1.0, dlogits=None):
    """Gradient of the routing weights with respect to the logits, the choice held fixed:
    ids int32 [T, k] and dweights float32 [T, k]; returns dlogits [T, E] of logits' type."""
    dt, T, E = _logits(logits)
    if ids.dim() != 2:
        raise ValueError("ids must be [T, k]")
    k = ids.shape[1]
    _check(ids, "ids", torch.int32, (T, k))
    _check(dweights, "dweights", torch.float32, (T, k))
    _same_device(logits, ids, dweights)
    dlogits = _given(dlogits, "dlogits", logits.dtype, (T, E), logits.device)
    st = _lib.load().f8f8bf16_route_backward(logits.data_ptr(), dt, ids.data_ptr(), dweights.data_ptr(), _score(score),
                                             1 if renormalize else 0, scale, dlogits.data_ptr(), T, E, k,
                                             _stream(logits.device))
    if st:
        _lib.layer_check(st, "f8f8bf16_route_backward")
    return dlogits


def _places(dst_row: torch.Tensor, T: int) -> int:
    if dst_row.dim() != 2:
        raise ValueError("dst_row must be [T, k]")
    k = dst_row.shape[1]
    _check(dst_row, "dst_row", torch.int32, (T, k))
    return k


def f8f8bf16_moe_dispatch(XQ, x_scale, dst_row, rows=None, XQs=None, xs_out=None):
    """Copies codes XQ [T, K] and scales x_scale ([T] or [T, K / 128]) to the experts'
    order: row dst_row[t, j] of the outputs is row t, for every j.  Returns (XQs
    [rows, K], xs_out), rows = T * k unless given; entries of dst_row outside
    [0, rows) are left out, rows that no entry names are not written."""
    XQ = _bytes(XQ, "XQ")
    T, K = _matrix(XQ, "XQ", torch.uint8, "[T, K]")
    dev = XQ.device
    k = _places(dst_row, T)
    if x_scale.dim() == 1:
        cols, tail = 1, ()
    elif x_scale.dim() == 2:
        cols = x_scale.shape[1]
        tail = (cols,)
    else:
        raise ValueError("x_scale must be [T] or [T, columns]")
    _check(x_scale, "x_scale", torch.float32, (T, *tail))
    _same_device(XQ, x_scale, dst_row)
    R = T * k if rows is None else rows
    XQs = _given(XQs, "XQs", torch.uint8, (R, K), dev)
    xs_out = _given(xs_out, "xs_out", torch.float32, (R, *tail), dev)
    st = _lib.load().f8f8bf16_moe_dispatch(XQ.data_ptr(), x_scale.data_ptr(), cols, dst_row.data_ptr(), XQs.data_ptr(),
                                           xs_out.data_ptr(), T, k, R, K, _stream(dev))
    if st:
        _lib.layer_check(st, "f8f8bf16_moe_dispatch")
    return XQs, xs_out


def f8f8bf16_moe_combine(Y, dst_row, weights=None, addend=None, out=None):
    """out[t] = sum_j weights[t, j] * Y[dst_row[t, j]] + addend[t]: Y [R, N] bf16, dst_row
    int32 [T, k], weights float32 [T, k] (None: ones), addend [T, N] bf16 or None.
    Returns out [T, N] bf16, which may be addend itself."""
    R, N = _matrix(Y, "Y", torch.bfloat16, "[R, N]")
    T = dst_row.shape[0]
    k = _places(dst_row, T)
    if weights is not None:
        _check(weights, "weights", torch.float32, (T, k))
    if addend is not None:
        _check(addend, "addend", torch.bfloat16, (T, N))
    _same_device(Y, dst_row, weights, addend)
    out = _given(out, "out", torch.bfloat16, (T, N), Y.device)
    st = _lib.load().f8f8bf16_moe_combine(Y.data_ptr(), dst_row.data_ptr(), _ptr(weights), _ptr(addend), out.data_ptr(),
                                          T, k, R, N, _stream(Y.device))
    if st:
        _lib.layer_check(st, "f8f8bf16_moe_combine")
    return out


def f8f8bf16_moe_combine_backward(dout, dst_row, weights=None, Y=None, rows=None, dY=None, dweights=None):
    """Gradients of combine: dout [T, N] bf16, Y [R, N] the forward's rows (None: no
    gradient of the weights, and rows gives R, T * k by default).  Returns (dY [R, N]
    bf16, dweights float32 [T, k] or None); rows of dY that no entry of dst_row names are
    not written.  With weights and Y None it is a dispatch of bf16 rows."""
    T, N = _matrix(dout, "dout", torch.bfloat16, "[T, N]")
    dev = dout.device
    k = _places(dst_row, T)
    if weights is not None:
        _check(weights, "weights", torch.float32, (T, k))
    if Y is not None:
        R = Y.shape[0] if Y.dim() == 2 else -1
        _check(Y, "Y", torch.bfloat16, (R, N))
        if rows is not None and rows != R:
            raise ValueError(f"rows={rows}, but Y has {R}")
        dweights = _given(dweights, "dweights", torch.float32, (T, k), dev)
    else:
        R = T * k if rows is None else rows
        if dweights is not None:
            raise ValueError("dweights needs Y")
    _same_device(dout, dst_row, weights, Y)
    dY = _given(dY, "dY", torch.bfloat16, (R, N), dev)
    st = _lib.load().f8f8bf16_moe_combine_backward(dout.data_ptr(), dst_row.data_ptr(), _ptr(weights), _ptr(Y),
                                                   dY.data_ptr(), _ptr(dweights), T, k, R, N, _stream(dev))
    if st:
        _lib.layer_check(st, "f8f8bf16_moe_combine_backward")
    return dY, dweights


def f8f8bf16_silu_mul_quantize(H, block=0, checkpoint=False, AQ=None, a_scale=None, HQ=None, h_scale=None) -> SiluMul:
    """silu(gate) * up of H = [gate | up] [rows, 2 I] bf16 with an fp8 output (block as in
    rmsnorm_quantize) and, with checkpoint=True (or HQ and h_scale given), the 8-bit
    checkpoint of H that silu_mul_backward reads.  Returns SiluMul(AQ [rows, I], a_scale,
    HQ [rows, 2 I] or None, h_scale [rows, 2, ceil(I / 128)] or None)."""
    rows, two = _matrix(H, "H", torch.bfloat16, "[rows, 2 I]")
    if two % 2:
        raise ValueError(f"H must have an even number of columns, got {two}")
    I = two // 2
    dev = H.device
    cols = _block_cols(block, I)
    AQ = _given(AQ, "AQ", torch.uint8, (rows, I), dev)
    a_scale = _given(a_scale, "a_scale", torch.float32, (rows, cols) if cols else (rows,), dev)
    if checkpoint or HQ is not None or h_scale is not None:
        HQ = _given(HQ, "HQ", torch.uint8, (rows, two), dev)
        h_scale = _given(h_scale, "h_scale", torch.float32, (rows, 2, (I + 127) // 128), dev)
    st = _lib.load().f8f8bf16_silu_mul_quantize(H.data_ptr(), block, AQ.data_ptr(), a_scale.data_ptr(), _ptr(HQ),
                                                _ptr(h_scale), rows, I, _stream(dev))
    if st:
        _lib.layer_check(st, "f8f8bf16_silu_mul_quantize")
    return SiluMul(AQ, a_scale, HQ, h_scale)


def f8f8bf16_silu_mul_backward(dA, HQ, h_scale, dH=None):
    """Gradient of silu(gate) * up from the 8-bit checkpoint: dA [rows, I] bf16; returns
    dH [rows, 2 I] bf16."""
    rows, I = _matrix(dA, "dA", torch.bfloat16, "[rows, I]")
    HQ = _bytes(HQ, "HQ")
    _check(HQ, "HQ", torch.uint8, (rows, 2 * I))
    _check(h_scale, "h_scale", torch.float32, (rows, 2, (I + 127) // 128))
    _same_device(dA, HQ, h_scale)
    dH = _given(dH, "dH", torch.bfloat16, (rows, 2 * I), dA.device)
    st = _lib.load().f8f8bf16_silu_mul_backward(dA.data_ptr(), HQ.data_ptr(), h_scale.data_ptr(), dH.data_ptr(), rows, I,
                                                _stream(dA.device))
    if st:
        _lib.layer_check(st, "f8f8bf16_silu_mul_backward")
    return dH


def f8f8bf16_k_offsets_capacity(R: int, G: int) -> int:
    """Columns that quantize_k_offsets needs for R rows in G groups."""
    return _lib.load().f8f8bf16_k_offsets_capacity(R, G)


def f8f8bf16_quantize_k_offsets(X, M_sizes, x_scale=None, XT=None, t_scale=None, k_offsets=None, workspace=None):
    """The weight gradient's operand from rows in expert order: X [R, K] bf16, or fp8
    codes with x_scale ([R] or [R, K / 128]); M_sizes int64 [G].  Returns (XT uint8
    [K, capacity], t_scale float32 [G, K], k_offsets int32 [G]), an operand of
    f8f8bf16_rowwise_grouped_k_offsets with its scales and offsets."""
    codes = x_scale is not None
    if codes:
        X = _bytes(X, "X")
    R, K = _matrix(X, "X", torch.uint8 if codes else torch.bfloat16, "[R, K]")
    dev = X.device
    if M_sizes.dim() != 1:
        raise ValueError("M_sizes must be [G]")
    G = M_sizes.shape[0]
    _check(M_sizes, "M_sizes", torch.int64, (G,))
    cols = 0
    if codes:
        cols = 1 if x_scale.dim() == 1 else K // 128
        _check(x_scale, "x_scale", torch.float32, (R,) if x_scale.dim() == 1 else (R, cols))
    _same_device(X, M_sizes, x_scale)
    lib = _lib.load()
    XT = _given(XT, "XT", torch.uint8, (K, lib.f8f8bf16_k_offsets_capacity(R, G)), dev)
    t_scale = _given(t_scale, "t_scale", torch.float32, (G, K), dev)
    k_offsets = _given(k_offsets, "k_offsets", torch.int32, (G,), dev)
    ws, size, _hold = _workspace(workspace, lib.f8f8bf16_quantize_k_offsets_workspace(R, G, K), dev)
    st = lib.f8f8bf16_quantize_k_offsets(X.data_ptr(), _lib.DTYPE_E4M3 if codes else _lib.DTYPE_BF16, _ptr(x_scale), cols,
                                         M_sizes.data_ptr(), XT.data_ptr(), t_scale.data_ptr(), k_offsets.data_ptr(), ws,
                                         size, R, G, K, _stream(dev))
    if st:
        _lib.layer_check(st, "f8f8bf16_quantize_k_offsets")
    return XT, t_scale, k_offsets
