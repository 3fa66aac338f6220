"""The router's choice by the oracle against the definition in 80-bit arithmetic (CPU)."""
import numpy as np
import pytest

from oracle import layer as L


def choice(x, k, b, score):
    """The k best experts of each row, in long double, ties to the lowest index."""
    x = x.astype(np.longdouble)
    if score == "sigmoid":
        p = 1 / (1 + np.exp(-x))
    else:
        e = np.exp(x - x.max(axis=1, keepdims=True))
        p = e / e.sum(axis=1, keepdims=True)
    return np.argsort(-(p + b), axis=1, kind="stable")[:, :k]


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_scores_far_below_the_largest_keep_their_order(score):
    rng = np.random.default_rng(1)
    x = rng.normal(-20, 12, (200, 64)).astype(np.float32)
    for bias in (None, np.zeros(64)):
        assert np.array_equal(L.route(x, 8, bias, score=score)[1], choice(x, 8, 0, score))


def test_sigmoids_near_one_keep_their_order():
    rng = np.random.default_rng(2)
    steps = rng.permuted(np.tile(np.arange(32), (64, 1)), axis=1).astype(np.float32)
    x = (np.float32(rng.uniform(8, 20, (64, 1))) + steps * np.float32(2.0 ** -19)).astype(np.float32)
    b = rng.choice([0.0, 0.25], 32)
    assert np.array_equal(L.route(x, 8, b, score="sigmoid")[1], choice(x, 8, b, "sigmoid"))


def test_groups_of_small_scores_keep_their_order():
    """Two experts per group: the best groups by the sums of softmax shares."""
    rng = np.random.default_rng(3)
    x = rng.normal(0, 15, (200, 16)).astype(np.float32)
    e = np.exp(x.astype(np.longdouble) - x.max(axis=1, keepdims=True))
    best = np.argsort(-e.reshape(200, 8, 2).sum(-1), axis=1, kind="stable")[:, :3]
    ids = L.route(x, 6, score="softmax", n_group=8, topk_group=3, group_top=2)[1]
    assert np.array_equal(np.sort(ids // 2, axis=1), np.sort(np.repeat(best, 2, axis=1), axis=1))


def test_significant_bits():
    for x in (1.0, 1 - 2.0 ** -53, 1 + 2.0 ** -52, 1 - 2.0 ** -50):
        assert L.significant(x) == 1.0
    assert L.significant(1 + 2.0 ** -43) == 1 + 2.0 ** -43 and L.significant(-3e-40) == pytest.approx(-3e-40, rel=2.0 ** -44)
    assert L.significant(0.0) == 0.0 and L.significant(1 + 2.0 ** -44) == 1 + 2.0 ** -43
