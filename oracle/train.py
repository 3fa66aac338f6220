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
# Of codes 0 to 126: eight subnormal ones, then eight to a power of two.
E4M3_MAGNITUDES = [(i % 8 + 8 * (i > 7)) * 2.0 ** (max(i // 8, 1) - 10) for i in range(127)]


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


def nearest(codes, v, amax):
    """Which e4m3 codes (uint8) are the nearest to v / s, s = max(amax, 2^-100) / 448, ties to the even one.  v and amax hold
    fp32 values: 448 |v| and a middle of two codes (5 bits) times amax have less than 53 bits, so both are exact here."""
    table = torch.tensor([E4M3_MAGNITUDES[i] for i in range(127)], dtype=torch.float64, device=v.device)
    i = (codes & 0x7F).long()
    amax = amax.clamp_min(2.0 ** -100)
    x, even = v.abs() * E4M3_MAX, i % 2 == 0
    here = table[i.clamp_max(126)]
    low = (here + table[(i - 1).clamp(0, 126)]) / 2 * amax
    high = torch.where(i < 126, (here + table[(i + 1).clamp_max(126)]) / 2 * amax, math.inf)
    sign = (codes >= 0x80) == (v < 0)
    return (i < 127) & ((x > low) | (x == low) & even | (i == 0)) & ((x < high) | (x == high) & even) & (sign | (i == 0))


def clip(grads, max_norm, eps):
    """(norm, factor, scaled gradients)."""
    norm = math.sqrt(math.fsum(float(v) for g in grads for v in g.double().flatten().square().split(1 << 16) for v in [v.sum()]))
    if math.isinf(max_norm) or norm + eps == 0:
        factor = 1.0
    else:
        factor = math.nan if math.isnan(norm) else min(1.0, max_norm / (norm + eps))
    return norm, factor, [g.double() * factor for g in grads]
