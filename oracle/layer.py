"""Plain CPU oracle of the layer operators (include/fp8gg_layer.h), in 64 bits.

TEST INFRASTRUCTURE.  Only the tests may import this module; the GPU library shares no
code with it.  Inputs are numpy arrays of the values themselves (float64, exactly what
the bf16 / e4m3 / fp32 tensors hold); results are the unrounded real ones, except where
a rounding is part of the definition (the residual sum, the codes' scales).
"""
from __future__ import annotations

import numpy as np

E4M3_MAX = 448.0
BLOCK = 128


def bf16(x: np.ndarray) -> np.ndarray:
    """float64 -> nearest bf16 (ties to even), as float64.  Inputs are sums of two bf16
    values or fp32 ones, finite."""
    x = np.asarray(x, np.float64)
    m, e = np.frexp(x)                                   # x = m 2^e, 0.5 <= |m| < 1
    step = np.exp2(np.maximum(e - 8, -133).astype(np.float64))
    return np.round(x / step) * step


def scale_of(amax: np.ndarray) -> np.ndarray:
    return np.where(amax > 0, np.maximum(amax, 2.0 ** -100) / E4M3_MAX, 1.0)


def block_amax(v: np.ndarray, block: int) -> np.ndarray:
    """Largest magnitudes: [rows] for block 0, else [rows, ceil(K / block)]."""
    a = np.abs(v)
    if not block:
        return a.max(axis=1, initial=0.0)
    K = v.shape[1]
    return np.stack([a[:, c:c + block].max(axis=1) for c in range(0, K, block)], axis=1)


def spread(s: np.ndarray, K: int) -> np.ndarray:
    """Scales [rows] or [rows, blocks] -> one per element [rows, K]."""
    if s.ndim == 1:
        return np.repeat(s[:, None], K, axis=1)
    return np.repeat(s, BLOCK, axis=1)[:, :K]


# -- norm -------------------------------------------------------------------

def rmsnorm(x, residual, weight, eps):
    """(h, y, rstd)."""
    h = x if residual is None else bf16(x + residual)
    rstd = 1.0 / np.sqrt((h * h).mean(axis=1) + eps)
    return h, h * rstd[:, None] * weight, rstd


def rmsnorm_backward(dy, h, weight, rstd, dresidual):
    """(dx, dweight)."""
    xhat = h * rstd[:, None]
    g = dy * weight
    dx = rstd[:, None] * (g - xhat * (g * xhat).mean(axis=1, keepdims=True))
    if dresidual is not None:
        dx = dx + dresidual
    return dx, (dy * xhat).sum(axis=0)


# -- routing ----------------------------------------------------------------

def _counted(x):
    x = np.where(np.isnan(x), -np.inf, x)
    return np.minimum(x, np.float64(np.finfo(np.float32).max))


def scores(x, score):
    if score == "sigmoid":
        with np.errstate(over="ignore"):
            return 1.0 / (1.0 + np.exp(-x))
    m = x.max(axis=1, keepdims=True)
    e = np.exp(x - np.where(np.isfinite(m), m, 0.0))
    s = e.sum(axis=1, keepdims=True)
    return e / np.where(s > 0, s, 1.0)


def shares(x, score):
    """Scores of the chosen logits over their sum, by way of their logarithms."""
    log = x if score == "softmax" else np.minimum(x, 0.0) - np.log1p(np.exp(-np.abs(x)))
    w = np.exp(log - log.max())
    return w / w.sum()


def significant(x, bits=44):
    """x rounded to so many significant bits, halves away from zero."""
    m, e = np.frexp(np.float64(x))
    return float(np.ldexp(np.trunc(m * 2.0 ** bits + np.copysign(0.5, m)), e - bits))


def route(logits, k, bias=None, score="softmax", n_group=1, topk_group=1, group_top=1, renormalize=True, scale=1.0):
    """(weights, ids): one token after the other, by sorting."""
    x = _counted(np.asarray(logits, np.float64))
    T, E = x.shape
    b = np.zeros(E) if bias is None else _counted(np.asarray(bias, np.float64))
    p = scores(x, score)
    weights, ids = np.zeros((T, k)), np.full((T, k), -1, np.int64)
    per = E // n_group
    for t in range(T):
        ok = (x[t] > -np.inf) & (b > -np.inf)
        sums = np.where(ok, p[t] + b, -np.inf)
        key = np.where(ok, x[t], -np.inf) if bias is None else sums       # p rises with x
        if n_group > 1:
            best = []
            for g in range(n_group):
                v = np.sort((key if group_top == 1 else sums)[g * per:(g + 1) * per])[::-1][:group_top]
                v = v[v > -np.inf]
                # sums that are equal in exact arithmetic tie
                best.append(-np.inf if not v.size else v[0] if group_top == 1 else significant(v.sum()))
            order = sorted(range(n_group), key=lambda g: (-best[g], g))
            kept = [g for g in order[:topk_group] if best[g] > -np.inf]
            key = np.where(np.isin(np.arange(E) // per, kept), key, -np.inf)
        order = sorted(range(E), key=lambda e: (-key[e], e))
        chosen = [e for e in order[:k] if key[e] > -np.inf]
        if not chosen:
            continue
        ids[t, :len(chosen)] = chosen
        w = shares(x[t, chosen], score) if renormalize else p[t, chosen]
        weights[t, :len(chosen)] = w * scale
    return weights, ids


def plan(ids, E):
    """(M_sizes, dst_row): a stable counting sort of the pairs."""
    flat = ids.reshape(-1)
    sizes = np.bincount(flat[flat >= 0], minlength=E).astype(np.int64)
    at = np.concatenate([[0], np.cumsum(sizes)[:-1]])
    dst = np.full(flat.shape, -1, np.int64)
    for i, e in enumerate(flat):
        if e >= 0:
            dst[i] = at[e]
            at[e] += 1
    return sizes, dst.reshape(ids.shape)


def route_backward(logits, ids, dweights, score="softmax", renormalize=True, scale=1.0):
    """(dlogits, size): the gradient and the sum of the magnitudes that it is made of."""
    x = _counted(np.asarray(logits, np.float64))
    dx, size = np.zeros_like(x), np.zeros_like(x)
    p = scores(x, score)
    for t in range(x.shape[0]):
        here = (ids[t] >= 0) & (ids[t] < x.shape[1])
        c, g = ids[t][here], dweights[t][here] * scale
        if renormalize:
            if c.size == 0:
                continue
            q = shares(x[t, c], score)
            f = q if score == "softmax" else q / (1.0 + np.exp(x[t, c]))
            dx[t, c] = f * (g - (q * g).sum())
            size[t, c] = f * (np.abs(g) + (q * np.abs(g)).sum())
        elif score == "sigmoid":
            dx[t, c] = g * p[t, c] / (1.0 + np.exp(x[t, c]))
            size[t, c] = np.abs(dx[t, c])
        else:
            d, da = (p[t, c] * g).sum(), (p[t, c] * np.abs(g)).sum()
            dx[t], size[t] = -p[t] * d, p[t] * da
            dx[t, c] += p[t, c] * g
            size[t, c] += p[t, c] * np.abs(g)
    return dx, size


# -- exchange ---------------------------------------------------------------

def dispatch(rows, dst, R):
    """(out [R, ...], written [R])."""
    out, written = np.zeros((R,) + rows.shape[1:], rows.dtype), np.zeros(R, bool)
    for t in range(dst.shape[0]):
        for r in dst[t]:
            if 0 <= r < R:
                out[r], written[r] = rows[t], True
    return out, written


def combine(y, dst, weights, addend):
    """(out, size): the sums and the sums of magnitudes."""
    T, k = dst.shape
    out = np.zeros((T, y.shape[1])) if addend is None else addend.copy()
    size = np.abs(out)
    for t in range(T):
        for j in range(k):
            if 0 <= dst[t, j] < y.shape[0]:
                w = 1.0 if weights is None else weights[t, j]
                out[t] += w * y[dst[t, j]]
                size[t] += np.abs(w * y[dst[t, j]])
    return out, size


def combine_backward(dout, dst, weights, y):
    """(dy, written, dweights, size)."""
    T, k = dst.shape
    dy, written = np.zeros_like(y), np.zeros(y.shape[0], bool)
    dw, size = np.zeros((T, k)), np.zeros((T, k))
    for t in range(T):
        for j in range(k):
            r = dst[t, j]
            if 0 <= r < y.shape[0]:
                dy[r] = dout[t] * (1.0 if weights is None else weights[t, j])
                written[r] = True
                dw[t, j] = (dout[t] * y[r]).sum()
                size[t, j] = np.abs(dout[t] * y[r]).sum()
    return dy, written, dw, size


# -- checkpoints ------------------------------------------------------------

def _sigmoid(g):
    with np.errstate(over="ignore"):
        return 1.0 / (1.0 + np.exp(-g))


def silu_mul(h):
    gate, up = np.split(h, 2, axis=1)
    return gate * _sigmoid(gate) * up


def silu_mul_backward(da, h):
    """(dh, size)."""
    gate, up = np.split(h, 2, axis=1)
    s = _sigmoid(gate)
    dg, du = da * up * s * (1.0 + gate * (1.0 - s)), da * gate * s
    sg = np.abs(da * up) * s * (1.0 + np.abs(gate) * (1.0 - s))
    return np.concatenate([dg, du], axis=1), np.concatenate([sg, np.abs(du)], axis=1)


def group_ends(sizes, R):
    """Row ends of the groups: negative counts are 0, ends are cut at R."""
    return np.minimum(np.cumsum(np.maximum(np.asarray(sizes, np.int64), 0)), R)


def k_offsets(v, sizes, cap):
    """(values / scale [K, cap], valid [cap], scales [G, K], offsets [G])."""
    R, K = v.shape
    out, valid = np.zeros((K, cap)), np.zeros(cap, bool)
    scales, offs, row, col = [], [], 0, 0
    for end in group_ends(sizes, R):
        part = v[row:end]
        s = scale_of(np.abs(part).max(axis=0, initial=0.0))
        out[:, col:col + end - row] = (part / s).T
        valid[col:col + end - row] = True
        col += -(-(end - row) // 16) * 16
        row = int(end)
        scales.append(s)
        offs.append(col)
    return out, valid, np.array(scales), np.array(offs, np.int64)
