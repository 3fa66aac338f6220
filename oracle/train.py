"""Plain oracle of the training operators (include/fp8gg_train.h), in 64 bits.

TEST INFRASTRUCTURE.  Only the tests may import this module; the GPU library shares no
code with it.  Inputs are float64 tensors of the values themselves, on any device; results
are the unrounded real ones.
"""
from __future__ import annotations

import math

import torch

from .layer import E4M3_MAX

BLOCK = 128


def group_rows(sizes, M: int) -> list[range]:
    """Rows of each group, the counts clamped: negative ones to 0, ends to M."""
    rows, at = [], 0
    for n in sizes:
        end = min(M, at + max(0, int(n)))
        rows.append(range(at, end))
        at = end
    return rows


def forward(x, w, sizes):
    """(Y, the sum of the products' magnitudes, which rows are written)."""
    return _rows(x, w.mT, sizes)


def dgrad(dy, w, sizes):
    return _rows(dy, w, sizes)


def _rows(p, q, sizes):
    M = p.shape[0]
    out = torch.zeros(M, q.shape[2], dtype=torch.float64, device=p.device)
    size = torch.zeros_like(out)
    written = torch.zeros(M, dtype=torch.bool)
    for g, r in enumerate(group_rows(sizes, M)):
        if len(r):
            s = slice(r.start, r.stop)
            out[s] = p[s] @ q[g]
            size[s] = p[s].abs() @ q[g].abs()
            written[s] = True
    return out, size, written


def wgrad(dy, x, sizes):
    """(dW, the sum of the products' magnitudes)."""
    rows = group_rows(sizes, dy.shape[0])
    parts = [(dy[r.start:r.stop].T.contiguous(), x[r.start:r.stop]) for r in rows]
    return torch.stack([d @ v for d, v in parts]), torch.stack([d.abs() @ v.abs() for d, v in parts])


def scale_of(amax):
    return torch.where(amax > 0, amax.clamp_min(2.0 ** -100) / E4M3_MAX, 1.0)


def row_blocks(x):
    """(values over their scales, scales) of rows in blocks of 128 columns."""
    rows, K = x.shape
    b = x.view(rows, K // BLOCK, BLOCK)
    s = scale_of(b.abs().amax(2))
    return (b / s[:, :, None]).view(rows, K), s


def weight_blocks(w):
    """(values over their scales, scales) of weights [G, N, K] in blocks of 128 x 128."""
    G, N, K = w.shape
    b = w.view(G, N // BLOCK, BLOCK, K // BLOCK, BLOCK)
    s = scale_of(b.abs().amax(4).amax(2))
    return (b / s[:, :, None, :, None]).view(G, N, K), s


def clip(grads, max_norm, eps):
    """(norm, factor, scaled gradients)."""
    norm = math.sqrt(math.fsum(float(v) for g in grads for v in g.double().flatten().square().split(1 << 16) for v in [v.sum()]))
    if math.isinf(max_norm) or norm + eps == 0:
        factor = 1.0
    else:
        factor = math.nan if math.isnan(norm) else min(1.0, max_norm / (norm + eps))
    return norm, factor, [g.double() * factor for g in grads]
