"""Comparisons of the layer operators with the 64-bit oracle.

u = 2^-24 is half a step of fp32, relative to the value.  Tolerances count roundings:
a bf16 result is off by half a step (2^-8 at most, relative) on top of the fp32 value
before it; a code by half a step of e4m3 (2^-4 relative, 2^-10 in the subnormal range,
in units of the scale) on top of the fp32 value before it.
"""
from __future__ import annotations

import numpy as np
import torch

import oracle

U = 2.0 ** -24
BF16 = 2.0 ** -8
GUARD = 256


def to_bf16(a: np.ndarray) -> torch.Tensor:
    """float array -> CPU bf16 tensor (values rounded)."""
    return torch.from_numpy(np.ascontiguousarray(a, np.float32)).to(torch.bfloat16)


def f64(t: torch.Tensor) -> np.ndarray:
    return t.detach().cpu().double().numpy()


def decode(codes: torch.Tensor) -> np.ndarray:
    return oracle.decode_e4m3fn(codes.cpu().numpy()).astype(np.float64)


def half_step(q: np.ndarray) -> np.ndarray:
    """Half the distance of neighbouring e4m3 values around q."""
    _, e = np.frexp(np.maximum(np.abs(q), 2.0 ** -6))
    return np.exp2((e - 1 - 4).astype(np.float64))


def assert_codes(codes: torch.Tensor, q: np.ndarray, rel: float, label: str = "") -> None:
    """codes stand for q (values over their scale) up to half a step, q known to rel."""
    got = decode(codes)
    assert np.all(np.isfinite(got)), f"{label}: {np.sum(~np.isfinite(got))} codes are NaN"
    tol = half_step(q * (1 + rel)) + np.abs(q) * rel
    bad = np.argwhere(np.abs(got - q) > tol)
    assert bad.size == 0, f"{label}: {len(bad)} codes off, first at {bad[0]}: {got[tuple(bad[0])]} for {q[tuple(bad[0])]}"


def assert_close(got: torch.Tensor, want: np.ndarray, tol: np.ndarray, label: str = "") -> None:
    g = f64(got)
    assert g.shape == want.shape, f"{label}: {g.shape} for {want.shape}"
    bad = np.argwhere(~(np.abs(g - want) <= tol))
    assert bad.size == 0, (f"{label}: {len(bad)} values off, first at {bad[0]}: {g[tuple(bad[0])]} for "
                           f"{want[tuple(bad[0])]}")


class Guarded:
    """An output of a given shape inside a larger buffer filled with a pattern."""

    def __init__(self, shape, dtype, fill=0xA5):
        n = int(np.prod(shape)) * torch.empty((), dtype=dtype).element_size()
        self.fill, self.n = fill, n
        self.whole = torch.full((n + 2 * GUARD,), fill, dtype=torch.uint8, device="cuda")
        self.t = self.whole[GUARD:GUARD + n].view(dtype).view(*shape)

    def check(self, label=""):
        w = self.whole.cpu().numpy()
        assert np.all(w[:GUARD] == self.fill), f"{label}: write before the buffer"
        assert np.all(w[GUARD + self.n:] == self.fill), f"{label}: write past the buffer"

    def untouched(self, rows) -> np.ndarray:
        """Which of the rows (first axis) still hold the pattern alone."""
        w = self.whole[GUARD:GUARD + self.n].view(self.t.shape[0], -1).cpu().numpy()
        return np.all(w[rows] == self.fill, axis=1)
