"""The training operators' oracle against loops over single values, autograd and planted mistakes (CPU)."""
import math

import pytest
import torch

from oracle import train as O


def case(seed=0, G=3, M=11, N=5, K=4):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g, dtype=torch.float64)  # noqa: E731
    return r(M, K), r(G, N, K), r(M, N), [4, 0, 6]


def test_group_rows():
    assert O.group_rows([3, -1, 2 ** 62, 5], 10) == [range(0, 3), range(3, 3), range(3, 10), range(10, 10)]
    assert O.group_rows([], 4) == [] and O.group_rows([0, 2], 4) == [range(0, 0), range(0, 2)]


def test_products_value_by_value():
    x, w, dy, s = case()
    y, size, written = O.forward(x, w, s)
    dx, _, _ = O.dgrad(dy, w, s)
    dw, wsize = O.wgrad(dy, x, s)
    group = [0] * 4 + [2] * 6 + [None]
    want_w = torch.zeros_like(w)
    for m, g in enumerate(group):
        assert bool(written[m]) == (g is not None)
        if g is None:
            continue
        for n in range(5):
            assert math.isclose(float(y[m, n]), sum(float(x[m, k] * w[g, n, k]) for k in range(4)), rel_tol=1e-12, abs_tol=1e-12)
            assert math.isclose(float(size[m, n]), sum(abs(float(x[m, k] * w[g, n, k])) for k in range(4)), rel_tol=1e-12)
            for k in range(4):
                want_w[g, n, k] += dy[m, n] * x[m, k]
        for k in range(4):
            assert math.isclose(float(dx[m, k]), sum(float(dy[m, n] * w[g, n, k]) for n in range(5)), rel_tol=1e-12, abs_tol=1e-12)
    assert torch.allclose(dw, want_w, rtol=1e-12, atol=1e-12) and bool((wsize >= dw.abs() - 1e-12).all())


def test_gradients_are_those_of_the_forward_product():
    x, w, dy, s = case(1)
    x.requires_grad_(True)
    w.requires_grad_(True)
    parts = [x[r.start:r.stop] @ w[g].T for g, r in enumerate(O.group_rows(s, 11))]
    gx, gw = torch.autograd.grad((torch.cat(parts) * dy[:10]).sum(), (x, w))
    assert torch.allclose(O.dgrad(dy, w.detach(), s)[0], gx) and torch.allclose(O.wgrad(dy, x.detach(), s)[0], gw)


@pytest.mark.parametrize("wrong", [[4, 1, 5], [3, 0, 7], [6, 0, 4]])
def test_a_shifted_boundary_is_seen(wrong):
    x, w, dy, s = case(2)
    assert not torch.allclose(O.forward(x, w, s)[0], O.forward(x, w, wrong)[0])
    assert not torch.allclose(O.wgrad(dy, x, s)[0], O.wgrad(dy, x, wrong)[0])


def test_blocks():
    w = torch.zeros(1, 256, 128, dtype=torch.float64)
    w[0, 130, 7] = -896.0
    w[0, 3, 5] = 2.0 ** -120
    q, s = O.weight_blocks(w)
    assert s.shape == (1, 2, 1) and float(s[0, 1, 0]) == 2.0 and float(s[0, 0, 0]) == 2.0 ** -100 / 448 and float(q[0, 130, 7]) == -448.0
    x = torch.zeros(2, 256, dtype=torch.float64)
    x[1, 200] = 4.48
    q, s = O.row_blocks(x)
    assert s.tolist()[0] == [1.0, 1.0] and math.isclose(float(s[1, 1]), 0.01) and math.isclose(float(q[1, 200]), 448.0)


def test_nearest_against_fractions():
    """Over single values in exact fractions, ties among them; and values on the wrong side of a middle are seen."""
    from fractions import Fraction
    table = [Fraction(m) for m in O.E4M3_MAGNITUDES]
    assert float(table[126]) == 448 and float(table[1]) == 2.0 ** -9 and sorted(table) == table
    g = torch.Generator().manual_seed(4)
    amax = torch.randint(128, 256, (400,), generator=g).double() / 128
    v = amax * 0 + torch.randint(-255, 256, (400,), generator=g).double() / 256 / torch.exp2(torch.randint(0, 12, (400,), generator=g).double())
    ties = 0
    for a, x in zip(amax.tolist(), v.tolist()):
        q = abs(Fraction(x)) * 448 / Fraction(a)
        off = [abs(q - t) for t in table]
        best = [i for i in range(127) if off[i] == min(off)]
        ties += len(best) > 1
        want = min(best, key=lambda i: i % 2)
        codes = torch.arange(256, dtype=torch.uint8)
        ok = O.nearest(codes, torch.full((256,), x, dtype=torch.float64), torch.tensor(a, dtype=torch.float64))
        signed = {want} | {want + 128} if want == 0 else {want + 128 * (x < 0)}
        assert set(ok.nonzero().flatten().tolist()) == signed, (a, x)
    assert ties


def test_values_rounded_before_their_codes_are_seen():
    """A code of v times the rounded 448 / amax, or of v over the rounded scale, is not always the nearest."""
    g = torch.Generator().manual_seed(5)
    amax = torch.randint(128, 256, (1 << 18,), generator=g).float() / 128
    v = torch.randint(128, 256, (1 << 18,), generator=g).float() / 256
    for q in (v * (448.0 / amax), v / (amax * (1.0 / 448.0)), v / (amax / 448.0)):
        codes = q.to(torch.float8_e4m3fn).view(torch.uint8)
        wrong = ~O.nearest(codes, v.double(), amax.double())
        assert 0 < int(wrong.sum()) < 1 << 13
    exact = (v.double() * 448 * 2.0 ** 40 / amax.double()).float() * 2.0 ** -40     # one rounding of the quotient: bf16's ties survive it
    assert bool(O.nearest(exact.to(torch.float8_e4m3fn).view(torch.uint8), v.double(), amax.double()).all())


def test_clip():
    a, b = torch.tensor([3.0]), torch.tensor([[0.0, 4.0]])
    norm, factor, out = O.clip([a, b], 1.0, 0.0)
    assert norm == 5.0 and factor == 0.2 and [o.tolist() for o in out] == [[0.6000000000000001], [[0.0, 0.8]]]
    assert O.clip([a, b], 10.0, 0.0)[1] == 1.0 and O.clip([a, b], 1.0, 5.0)[1] == 0.1 and O.clip([], 1.0, 1e-6)[0] == 0.0


def test_clip_where_the_quotient_is_none():
    """An infinite bound and a norm of 0 without eps leave every value; an infinite norm under a bound gives 0, a NaN one NaN."""
    inf, nan = math.inf, math.nan
    for bad in (inf, -inf, nan):
        _, factor, out = O.clip([torch.tensor([1.0, bad])], inf, 0.0)
        assert factor == 1.0 and out[0][0] == 1.0
    assert O.clip([torch.zeros(3)], 0.0, 0.0)[1] == 1.0
    assert not O.clip([torch.zeros(3)], 0.0, 0.0)[2][0].any()
    _, factor, out = O.clip([torch.tensor([1.0, inf])], 2.0, 0.0)
    assert factor == 0.0 and out[0][0] == 0.0 and out[0][1].isnan()
    assert math.isnan(O.clip([torch.tensor([1.0, nan])], 2.0, 0.0)[1])
