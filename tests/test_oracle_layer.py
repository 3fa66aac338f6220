"""Pins of the layer operators' oracle: closed forms, numeric differences, invariants
and planted mistakes (CPU)."""
import numpy as np
import pytest

from oracle import layer as L


def test_bf16_rounding_matches_torch():
    import torch
    rng = np.random.default_rng(1)
    x = (rng.normal(0, 1, 20000) * 2.0 ** rng.uniform(-30, 30, 20000)).astype(np.float32)
    x = np.concatenate([x, np.float32([1 + 2 ** -8, 1 + 3 * 2 ** -8, 1 + 2 ** -8 + 2 ** -20, 0.0, -0.0])])
    assert np.array_equal(L.bf16(x.astype(np.float64)), torch.from_numpy(x).to(torch.bfloat16).double().numpy())


def test_norm_of_constant_rows_is_the_weight():
    w = np.linspace(-2, 2, 16)
    h, y, rstd = L.rmsnorm(np.full((3, 16), 4.0), None, w, 0.0)
    assert np.allclose(y, w[None], rtol=1e-14) and np.allclose(rstd, 0.25, rtol=1e-14)


def differences(f, x, d, step=1e-6):
    """Directional derivative of f at x along d, by central differences."""
    return (f(x + step * d) - f(x - step * d)) / (2 * step)


def test_norm_gradient_against_differences():
    rng = np.random.default_rng(2)
    x, w, dy = rng.normal(0, 1, (4, 24)), rng.normal(1, 0.2, 24), rng.normal(0, 1, (4, 24))
    _, _, rstd = L.rmsnorm(x, None, w, 1e-3)
    dx, dw = L.rmsnorm_backward(dy, x, w, rstd, None)
    for _ in range(4):
        d, dd = rng.normal(0, 1, x.shape), rng.normal(0, 1, w.shape)
        assert np.isclose((dx * d).sum(), differences(lambda v: (L.rmsnorm(v, None, w, 1e-3)[1] * dy).sum(), x, d), rtol=1e-6)
        assert np.isclose((dw * dd).sum(), differences(lambda v: (L.rmsnorm(x, None, v, 1e-3)[1] * dy).sum(), w, dd), rtol=1e-6)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renormalize", [True, False])
def test_route_gradient_against_differences(score, renormalize):
    rng = np.random.default_rng(3)
    x = rng.normal(0, 1, (5, 12))
    weights, ids = L.route(x, 3, score=score, renormalize=renormalize, scale=1.7)
    dw = rng.normal(0, 1, weights.shape)
    dx, size = L.route_backward(x, ids, dw, score, renormalize, 1.7)
    assert np.all(size >= np.abs(dx) * (1 - 1e-12))

    def loss(v):   # the choice held fixed
        p = L.scores(v, score)
        w = np.take_along_axis(p, ids, 1)
        w = w / w.sum(1, keepdims=True) if renormalize else w
        return (w * 1.7 * dw).sum()
    for _ in range(4):
        d = rng.normal(0, 1, x.shape)
        assert np.isclose((dx * d).sum(), differences(loss, x, d), rtol=1e-6)


def test_route_ties_masks_groups():
    x = np.zeros((4, 8))
    x[1, 5] = 1.0
    x[2] = -np.inf
    x[3, :] = -np.inf
    x[3, 6], x[3, 2] = np.nan, 3.0
    w, ids = L.route(x, 2)
    assert ids.tolist() == [[0, 1], [5, 0], [-1, -1], [2, -1]]
    assert np.allclose(w[0], 0.5) and np.all(w[2] == 0) and w[3].tolist() == [1.0, 0.0]
    # the bias chooses, the weights come from the scores
    b = np.zeros(8)
    b[7] = 10.0
    w, ids = L.route(x[:1], 2, bias=b, renormalize=False)
    assert ids.tolist() == [[7, 0]] and np.allclose(w, 1 / 8)
    # groups of two: the pair 2, 3 has the best sum, the pair 6, 7 the best single one
    g = np.array([[0.0, 0.0, 2.0, 2.0, 0.0, 0.0, 3.0, -9.0]])
    assert L.route(g, 2, score="sigmoid", n_group=4, topk_group=1, group_top=2)[1].tolist() == [[2, 3]]
    assert L.route(g, 2, score="sigmoid", n_group=4, topk_group=1, group_top=1)[1].tolist() == [[6, 7]]


def test_sums_that_are_equal_in_exact_arithmetic_tie():
    """sigmoid(x) + sigmoid(-x) = 1 for every x: the groups tie, the lowest one stays."""
    x = np.array([[0.0, 0.0, -9.0, -9.0, 2.0, -2.0, 1.0, -1.0, 3.0, -3.0]])
    assert L.route(x[:, 4:], 1, score="sigmoid", n_group=3, topk_group=1, group_top=2)[1].tolist() == [[0]]
    assert L.route(x, 1, score="sigmoid", n_group=5, topk_group=1, group_top=2)[1].tolist() == [[0]]


def test_plan_is_a_stable_sort():
    rng = np.random.default_rng(4)
    ids = rng.integers(-1, 5, (40, 3))
    sizes, dst = L.plan(ids, 5)
    flat, d = ids.reshape(-1), dst.reshape(-1)
    order = np.argsort(np.where(flat < 0, 99, flat), kind="stable")[:int((flat >= 0).sum())]
    assert np.array_equal(d[order], np.arange(order.size)) and np.all(d[flat < 0] == -1)
    assert sizes.tolist() == [int((flat == e).sum()) for e in range(5)]


def test_exchange_gradients_against_differences():
    rng = np.random.default_rng(5)
    y, w, dout = rng.normal(0, 1, (7, 8)), rng.normal(0, 1, (3, 2)), rng.normal(0, 1, (3, 8))
    dst = np.array([[0, 3], [-1, 5], [6, 9]])
    dy, written, dw, _ = L.combine_backward(dout, dst, w, y)
    assert written.tolist() == [True, False, False, True, False, True, True]
    d, e = rng.normal(0, 1, y.shape), rng.normal(0, 1, w.shape)
    assert np.isclose((dy * d).sum(), differences(lambda v: (L.combine(v, dst, w, None)[0] * dout).sum(), y, d), rtol=1e-6)
    assert np.isclose((dw * e).sum(), differences(lambda v: (L.combine(y, dst, v, None)[0] * dout).sum(), w, e), rtol=1e-6)


def test_silu_gradient_against_differences():
    rng = np.random.default_rng(6)
    h, da = rng.normal(0, 2, (3, 20)), rng.normal(0, 1, (3, 10))
    dh, size = L.silu_mul_backward(da, h)
    assert np.all(size >= np.abs(dh) * (1 - 1e-12))
    for _ in range(4):
        d = rng.normal(0, 1, h.shape)
        assert np.isclose((dh * d).sum(), differences(lambda v: (L.silu_mul(v) * da).sum(), h, d), rtol=1e-6)


def test_k_offsets_layout():
    v = np.arange(1, 41, dtype=np.float64).reshape(20, 2)
    q, valid, s, offs = L.k_offsets(v, [3, 0, 17, 5], 64)
    assert offs.tolist() == [16, 16, 48, 48]           # the last group starts past the rows
    assert np.flatnonzero(valid).tolist() == [0, 1, 2] + list(range(16, 33))
    assert np.allclose(q[:, 0] * s[0], v[0]) and np.allclose(q[:, 32] * s[2], v[19])
    assert np.all(s[1] == 1) and np.all(s[3] == 1) and np.isclose(q[:, 2].max(), 448)


def test_planted_mistakes_are_seen():
    """Small changes of the definitions leave the tolerances used on the GPU."""
    rng = np.random.default_rng(7)
    h, da = rng.normal(0, 2, (3, 20)), rng.normal(0, 1, (3, 10))
    dh, size = L.silu_mul_backward(da, h)
    gate, up = np.split(h, 2, axis=1)
    s = 1 / (1 + np.exp(-gate))
    wrong = da * up * s * (1 + gate * s)               # s for 1 - s
    assert np.any(np.abs(wrong - dh[:, :10]) > 2.0 ** -8 * np.abs(dh[:, :10]) + 2.0 ** -16 * size[:, :10])
    x = rng.normal(0, 1, (4, 24))
    dx, _ = L.rmsnorm_backward(x, x, np.ones(24), 1 / np.sqrt((x * x).mean(1)), None)
    assert np.all(np.abs(dx) < 1e-12)                  # the norm is constant along its own row
