"""GPU parity of the bf16 products by group with the 64-bit oracle.

A sum of L products is formed in fp32: every addition rounds by half a step (2^-24) of what
it gives, which no order of additions makes larger than the sum S of the products'
magnitudes, and a product of two bf16 values is exact.  L + 8 such roundings (those of the
parts' sums among them) bound the error by (L + 8) 2^-24 S; a bf16 result is off by another
half step, 2^-8 relative.
"""
import pytest
import torch

from oracle import train as O
from tests import layer_parity as P

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def F():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    import fp8_rowwise_scaled_amd as F
    F.load()
    return F


def randn(g, *shape, sigma=1.0):
    return (torch.randn(*shape, generator=g, device="cuda") * sigma).to(torch.bfloat16)


def inputs(G, M, N, K, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed + G + M + N + K)
    return randn(g, M, K), randn(g, G, N, K, sigma=K ** -0.5 if K else 1.0), randn(g, M, N, sigma=0.1)


def sizes_of(G, M, how):
    """Counts: even, skewed with empty groups, all in one group, fewer than the rows, or not to be trusted."""
    g = torch.Generator().manual_seed(G * 31 + M)
    if how == "one":
        s = [0] * G
        s[G // 2] = M
    elif how == "wrong":
        s = [M // 3, -5, 2 ** 62, 7] + [2 ** 40] * G
        s = s[:G]
    else:
        p = torch.rand(G, generator=g, dtype=torch.float64) ** (4 if how != "even" else 0)
        p[torch.rand(G, generator=g) < (0.2 if how != "even" else 0.0)] = 0
        cut = (torch.cumsum(p, 0) / p.sum().clamp_min(1e-9) * (M if how != "short" else M * 2 // 3)).round().long().tolist()
        s = [b - a for a, b in zip([0] + cut, cut)]
    return s


def dev(s):
    return torch.tensor(s, dtype=torch.int64, device="cuda")


def check(got, want, size, L, bf16, label):
    tol = (L + 8) * 2.0 ** -24 * size + (2.0 ** -8 * want.abs() if bf16 else 0)
    bad = ~((got.double() - want).abs() <= tol)
    assert not bool(bad.any()), f"{label}: {int(bad.sum())} values off, first at {bad.nonzero()[0].tolist()}"


# sizes on all sides of the tiles (32, 128, 256 rows; 32, 64, 128, 256 columns; 32 and 64 of a contraction)
SHAPES = [
    (1, 1, 8, 8), (1, 1, 7168, 128), (3, 5, 16, 24), (8, 1, 256, 2048), (4, 33, 40, 72), (2, 64, 136, 8),
    (40, 700, 1048, 136), (9, 300, 1000, 264), (5, 650, 264, 520), (130, 400, 2056, 64), (70, 2100, 512, 200),
    (2, 520, 264, 328), (1, 257, 8, 64), (3, 1300, 1096, 896), (2, 900, 4104, 48), (6, 5000, 768, 136),
    (2, 9000, 2056, 64), (3, 9000, 40, 2312),
]


@pytest.mark.parametrize("G,M,N,K", SHAPES)
@pytest.mark.parametrize("how", ["even", "skewed", "one", "short", "wrong"])
def test_products(F, G, M, N, K, how):
    print(f"case products G={G} M={M} N={N} K={K} {how}", flush=True)
    x, w, dy = inputs(G, M, N, K)
    s = sizes_of(G, M, how)
    for name, args, width, L, oracle in (("forward", (x, w), N, K, O.forward), ("dgrad", (dy, w), K, N, O.dgrad)):
        out = P.Guarded((M, width), torch.bfloat16)
        if name == "forward":
            F.bf16_grouped_stacked(*args, dev(s), Y=out.t)
        else:
            F.bf16_grouped_stacked_dgrad(*args, dev(s), dX=out.t)
        torch.cuda.synchronize()
        out.check(name)
        want, size, written = oracle(args[0].double(), args[1].double(), s)
        check(out.t[written], want[written], size[written], L, True, name)
        assert out.untouched((~written).numpy()).all(), f"{name}: a row past the groups' end was written"
    want, size = O.wgrad(dy.double(), x.double(), s)
    for dtype in (torch.float32, torch.bfloat16):
        out = P.Guarded((G, N, K), dtype)
        F.bf16_grouped_stacked_wgrad(dy, x, dev(s), dW=out.t)
        torch.cuda.synchronize()
        out.check("wgrad")
        check(out.t, want, size, M, dtype is torch.bfloat16, f"wgrad {dtype}")
    held = torch.randn(G, N, K, device="cuda")
    out = held.clone()
    F.bf16_grouped_stacked_wgrad(dy, x, dev(s), dW=out, accumulate=True)
    check(out, want + held.double(), size + held.double().abs(), M, False, "wgrad accumulated")


# tiles over several rounds of the compute units, the last of them whole, in halves or in quarters, for small
# and large groups, and contractions that groups start at different places
@pytest.mark.parametrize("G,M,N,K", [
    (24, 1500, 2056, 256), (20, 600, 4104, 192), (67, 3000, 1280, 1024), (9, 1000, 2056, 64), (33, 700, 640, 4104),
    (1, 4096, 2056, 128), (1, 1024, 2048, 64), (3, 6000, 2312, 128), (2, 5000, 264, 2568), (5, 3000, 192, 4360)])
@pytest.mark.parametrize("how", ["even", "skewed", "short"])
def test_products_in_rounds(F, G, M, N, K, how):
    print(f"case rounds G={G} M={M} N={N} K={K} {how}", flush=True)
    x, w, dy = inputs(G, M, N, K, seed=3)
    s = sizes_of(G, M, how)
    for name, call, args, width, L, oracle in (("forward", F.bf16_grouped_stacked, (x, w), N, K, O.forward),
                                               ("dgrad", F.bf16_grouped_stacked_dgrad, (dy, w), K, N, O.dgrad)):
        out = P.Guarded((M, width), torch.bfloat16)
        call(*args, dev(s), **{"Y" if name == "forward" else "dX": out.t})
        torch.cuda.synchronize()
        out.check(name)
        want, size, written = oracle(args[0].double(), args[1].double(), s)
        check(out.t[written], want[written], size[written], L, True, name)
        assert out.untouched((~written).numpy()).all(), f"{name}: a row past the groups' end was written"


# the weights' gradient likewise: the groups' tiles over several rounds, in every XCD's eighths from 64 tiles a group on,
# of more groups than a wave has lanes
@pytest.mark.parametrize("G,M,N,K", [(6, 3000, 2056, 2056), (70, 2100, 2056, 2056), (130, 3000, 1800, 2312), (3, 700, 5128, 1032), (70, 4100, 520, 776)])
@pytest.mark.parametrize("how", ["even", "skewed", "one", "short", "wrong"])
def test_wgrad_in_rounds(F, G, M, N, K, how):
    print(f"case wgrad rounds G={G} M={M} N={N} K={K} {how}", flush=True)
    from fp8_rowwise_scaled_amd import _lib
    assert _lib.load().bf16_grouped_stacked_wgrad_workspace(G, M, N, K) == 0          # whole groups, no parts
    x, _, dy = inputs(G, M, N, K, seed=7)
    s = sizes_of(G, M, how)
    want, size = O.wgrad(dy.double(), x.double(), s)
    for dtype in (torch.float32, torch.bfloat16):
        out = P.Guarded((G, N, K), dtype)
        F.bf16_grouped_stacked_wgrad(dy, x, dev(s), dW=out.t)
        torch.cuda.synchronize()
        out.check("wgrad")
        check(out.t, want, size, M, dtype is torch.bfloat16, f"wgrad {dtype}")
    out = P.Guarded((G, N, K), torch.float32)
    held = torch.randn(G, N, K, device="cuda")
    out.t.copy_(held)
    for _ in range(2):                                    # twice over: two micro-batches
        F.bf16_grouped_stacked_wgrad(dy, x, dev(s), dW=out.t, accumulate=True)
    torch.cuda.synchronize()
    out.check("wgrad accumulated")
    check(out.t, 2 * want + held.double(), 2 * size + held.double().abs(), 2 * M, False, "wgrad accumulated")
    for g, r in enumerate(O.group_rows(s, M)):
        assert len(r) or torch.equal(out.t[g], held[g]), f"group {g} has no rows"


def columns(n):
    """Of 2^22: some at its start, across its middle and at its end; everything that a sum's order could move."""
    return torch.cat([torch.arange(40), torch.arange(n // 2 - 30, n // 2 + 50), torch.arange(n - 300, n)]).cuda()


@pytest.mark.parametrize("M,other", [(3, 16), (100, 64), (100, 264), (260, 264), (260, 8)])
def test_the_widest_rows(F, M, other):
    """N or K of 2^22, the most that the offsets of a tile's 256 rows hold in 32 bits.  A contraction that long has zeros but
    in a few places, which add nothing and no rounding: its length counts as theirs."""
    n = 1 << 22
    g = torch.Generator(device="cuda").manual_seed(M + other)
    at = columns(n)
    s = dev([M])
    wide = torch.zeros(M, n, dtype=torch.bfloat16, device="cuda")
    wide[:, at] = randn(g, M, len(at))
    w = torch.zeros(1, other, n, dtype=torch.bfloat16, device="cuda")
    w[0][:, at] = randn(g, other, len(at))
    narrow = randn(g, M, other)
    print(f"case widest rows M={M} other={other}", flush=True)
    xs, ws, ns = wide[:, at].double(), w[0][:, at].double(), narrow.double()
    y = F.bf16_grouped_stacked(wide, w, s)                              # K = 2^22
    check(y, xs @ ws.T, xs.abs() @ ws.abs().T, len(at), True, "forward, K")
    dx = F.bf16_grouped_stacked_dgrad(narrow, w, s)
    check(dx[:, at], ns @ ws, ns.abs() @ ws.abs(), other, True, "dgrad, K")
    assert int(dx.count_nonzero()) == int(dx[:, at].count_nonzero())
    for dtype in (torch.float32, torch.bfloat16):
        dw = F.bf16_grouped_stacked_wgrad(narrow, wide, s, dtype=dtype)[0]
        check(dw[:, at], ns.T @ xs, ns.abs().T @ xs.abs(), M, dtype is torch.bfloat16, "wgrad, K")
        assert int(dw.count_nonzero()) == int(dw[:, at].count_nonzero())
    w = w.transpose(1, 2).contiguous()
    y = F.bf16_grouped_stacked(narrow, w, s)                            # N = 2^22
    check(y[:, at], ns @ ws, ns.abs() @ ws.abs(), other, True, "forward, N")
    assert int(y.count_nonzero()) == int(y[:, at].count_nonzero())
    dx = F.bf16_grouped_stacked_dgrad(wide, w, s)
    check(dx, xs @ ws.T, xs.abs() @ ws.abs().T, len(at), True, "dgrad, N")
    for dtype in (torch.float32, torch.bfloat16):
        dw = F.bf16_grouped_stacked_wgrad(wide, narrow, s, dtype=dtype)[0]
        check(dw[at], xs.T @ ns, xs.abs().T @ ns.abs(), M, dtype is torch.bfloat16, "wgrad, N")
        assert int(dw.count_nonzero()) == int(dw[at].count_nonzero())


@pytest.mark.parametrize("G,M,N,K", [(1, 12000, 128, 72), (2, 5003, 264, 136), (3, 40000, 8, 8)])
def test_wgrad_in_parts(F, G, M, N, K):
    """Few tiles and many rows: the rows are split, also where a group has fewer than the others' parts."""
    from fp8_rowwise_scaled_amd import _lib
    assert _lib.load().bf16_grouped_stacked_wgrad_workspace(G, M, N, K) > 0
    x, _, dy = inputs(G, M, N, K)
    for how in ("even", "skewed", "one"):
        s = sizes_of(G, M, how)
        want, size = O.wgrad(dy.double(), x.double(), s)
        got = [F.bf16_grouped_stacked_wgrad(dy, x, dev(s), dtype=t) for t in (torch.float32, torch.bfloat16)]
        check(got[0], want, size, M, False, how)
        check(got[1], want, size, M, True, how)
        held = torch.randn_like(got[0])
        out = F.bf16_grouped_stacked_wgrad(dy, x, dev(s), dW=held.clone(), accumulate=True)
        check(out, want + held.double(), size + held.double().abs(), M, False, how)


@pytest.mark.parametrize("M,N,K", [(7, 64, 0), (7, 0, 64), (0, 64, 64), (300, 8, 0)])
def test_empty_axes(F, M, N, K):
    x, w, dy = inputs(2, M, N, K)
    s = dev([M // 2, M - M // 2])
    y = F.bf16_grouped_stacked(x, w, s)
    assert y.shape == (M, N) and not y.any()
    dx = F.bf16_grouped_stacked_dgrad(dy, w, s)
    assert dx.shape == (M, K) and not dx.any()
    dw = F.bf16_grouped_stacked_wgrad(dy, x, s)
    assert dw.shape == (2, N, K) and not dw.any()
    none = F.bf16_grouped_stacked(x, w[:0], s[:0], Y=torch.full((M, N), 3.0, dtype=torch.bfloat16, device="cuda"))
    assert bool((none == 3).all()) and F.bf16_grouped_stacked_wgrad(dy, x, s[:0]).shape == (0, N, K)


@pytest.mark.parametrize("G,M,N,K", [(4, 40, 136, 72), (3, 500, 264, 136), (2, 900, 1032, 200), (6, 5000, 768, 136)])
def test_infinities_and_nan_stay_where_they_belong(F, G, M, N, K):
    """Rows past the groups' end, other groups' rows and weights, and other rows of a tile hold NaN and
    infinities: whatever does not depend on them has the bits that it has without them."""
    x, w, dy = inputs(G, M, N, K)
    s = sizes_of(G, M, "short")
    used = sum(s)
    g = max(range(G), key=lambda i: s[i])
    first = sum(s[:g])
    clean = [F.bf16_grouped_stacked(x, w, dev(s)), F.bf16_grouped_stacked_dgrad(dy, w, dev(s)), F.bf16_grouped_stacked_wgrad(dy, x, dev(s))]
    nan, inf = float("nan"), float("inf")
    bad = first + s[g] // 2                               # one row of the largest group
    x2, dy2, w2 = x.clone(), dy.clone(), w.clone()
    for t in (x2, dy2):
        t[used:] = nan
        t[bad, ::2] = inf
        t[bad, 1::2] = nan
    y, dx, dw = F.bf16_grouped_stacked(x2, w, dev(s)), F.bf16_grouped_stacked_dgrad(dy2, w, dev(s)), F.bf16_grouped_stacked_wgrad(dy2, x2, dev(s))
    others = torch.ones(used, dtype=torch.bool, device="cuda")
    others[bad] = False
    for a, b in ((y, clean[0]), (dx, clean[1])):
        assert torch.equal(a[:used][others].view(torch.int16), b[:used][others].view(torch.int16))
        assert bool(a[bad].isnan().any())
    for e in range(G):
        # infinity times infinity, the even places of both, is infinite; every other place of the group NaN
        assert torch.equal(dw[e], clean[2][e]) if e != g else not bool(dw[e].isfinite().any())
    w2[g] = nan
    y, dx = F.bf16_grouped_stacked(x, w2, dev(s)), F.bf16_grouped_stacked_dgrad(dy, w2, dev(s))
    mine = torch.zeros(used, dtype=torch.bool, device="cuda")
    mine[first:first + s[g]] = True
    for a, b in ((y, clean[0]), (dx, clean[1])):
        assert torch.equal(a[:used][~mine].view(torch.int16), b[:used][~mine].view(torch.int16)) and bool(a[:used][mine].isnan().all())


def test_a_column_of_infinities(F):
    """... and of one row of the weights: one column of the output."""
    x, w, dy = inputs(2, 300, 136, 72)
    s = dev([150, 150])
    y = F.bf16_grouped_stacked(x, w, s)
    w[0, 5] = float("inf")
    z = F.bf16_grouped_stacked(x, w, s)
    keep = torch.ones(136, dtype=torch.bool, device="cuda")
    keep[5] = False
    assert torch.equal(z[:, keep], y[:, keep]) and torch.equal(z[150:], y[150:]) and not bool(z[:150, 5].isfinite().any())


def test_offsets_past_31_bits(F):
    """Weights and their gradients of more than 2^31 values, and rows of more."""
    G, N, K = 3, 32768, 32776
    g = torch.Generator(device="cuda").manual_seed(5)
    w = torch.zeros(G, N, K, dtype=torch.bfloat16, device="cuda")
    w[2, -40:] = randn(g, 40, K, sigma=0.01)
    x, dy = randn(g, 5, K), torch.zeros(5, N, dtype=torch.bfloat16, device="cuda")
    dy[:, -40:] = randn(g, 5, 40)
    s = [1, 1, 3]
    y = F.bf16_grouped_stacked(x, w, dev(s))
    want = x[2:].double() @ w[2, -40:].double().T
    check(y[2:, -40:], want, x[2:].double().abs() @ w[2, -40:].double().abs().T, K, True, "forward")
    assert not y[:2].any() and not y[2:, :-40].any()
    dx = F.bf16_grouped_stacked_dgrad(dy, w, dev(s))
    check(dx[2:], dy[2:, -40:].double() @ w[2, -40:].double(), dy[2:, -40:].double().abs() @ w[2, -40:].double().abs(), N, True, "dgrad")
    assert not dx[:2].any()
    dw = F.bf16_grouped_stacked_wgrad(dy, x, dev(s), dW=w)
    want = dy[2:, -40:].double().T @ x[2:].double()
    check(dw[2, -40:], want, dy[2:, -40:].double().abs().T @ x[2:].double().abs(), 5, True, "wgrad")
    assert not dw[2, :-40].any()
    del w, dw, y, dx
    M, K = 70000, 32776                                   # rows of more than 2^31 values
    x = torch.zeros(M, K, dtype=torch.bfloat16, device="cuda")
    x[-300:] = randn(g, 300, K)
    w = randn(g, 1, 16, K, sigma=0.01)
    y = F.bf16_grouped_stacked(x, w, dev([M]))
    check(y[-300:], x[-300:].double() @ w[0].double().T, x[-300:].double().abs() @ w[0].double().abs().T, K, True, "rows")
    assert not y[:-300].any()
    dy = torch.zeros(M, 16, dtype=torch.bfloat16, device="cuda")
    dy[-300:] = randn(g, 300, 16)
    dx = F.bf16_grouped_stacked_dgrad(dy, w, dev([M]), dX=torch.empty_like(x))
    check(dx[-300:], dy[-300:].double() @ w[0].double(), dy[-300:].double().abs() @ w[0].double().abs(), 16, True, "rows' gradient")
    assert not dx[:-300].any()


def test_results_do_not_depend_on_the_run(F):
    x, w, dy = inputs(6, 3000, 1032, 520)
    s = dev(sizes_of(6, 3000, "skewed"))
    first = [F.bf16_grouped_stacked(x, w, s), F.bf16_grouped_stacked_dgrad(dy, w, s), F.bf16_grouped_stacked_wgrad(dy, x, s)]
    for _ in range(3):
        again = [F.bf16_grouped_stacked(x, w, s), F.bf16_grouped_stacked_dgrad(dy, w, s), F.bf16_grouped_stacked_wgrad(dy, x, s)]
        assert all(torch.equal(a, b) for a, b in zip(first, again))


# all three kernels of the rows' products, tiles whole, in halves and in quarters
@pytest.mark.parametrize("G,M,N,K", [(3, 40, 136, 520), (24, 1500, 2056, 256), (20, 600, 1032, 4096), (2, 5000, 264, 2568), (3, 6000, 2312, 128), (9, 300, 1000, 264)])
def test_a_row_has_the_same_bits_wherever_it_lies(F, G, M, N, K):
    """At the same G, total_M, N and K: in another place of its group, among other rows and other groups' sizes.  The weights'
    gradient of a group: whatever the other groups hold, and wherever its own rows start."""
    print(f"case places G={G} M={M} N={N} K={K}", flush=True)
    x, w, dy = inputs(G, M, N, K)
    s = sizes_of(G, M, "even")
    y, dx, dw = F.bf16_grouped_stacked(x, w, dev(s)), F.bf16_grouped_stacked_dgrad(dy, w, dev(s)), F.bf16_grouped_stacked_wgrad(dy, x, dev(s))
    r = torch.Generator().manual_seed(M)
    for seed in range(3):
        other, _, dother = inputs(G, M, N, K, seed=20 + seed)
        # groups take rows from their neighbours on one side and lose some to the other, by up to half their size
        cut = [0]
        for g in range(G - 1):
            cut.append(min(M, max(cut[-1], sum(s[:g + 1]) + int(torch.randint(-(s[g] // 2), s[g] // 2 + 1, (1,), generator=r)))))
        t = [b - a for a, b in zip(cut, cut[1:] + [M])]
        rows = []                                         # (place now, place before) of the rows that are kept
        for g in range(G):
            n = min(s[g], t[g])
            now, before = (torch.randperm(k, generator=r)[:n] for k in (t[g], s[g]))
            rows.append(torch.stack([now + sum(t[:g]), before + sum(s[:g])]))
        now, before = torch.cat(rows, 1).cuda()
        other[now], dother[now] = x[before], dy[before]
        for got, want in ((F.bf16_grouped_stacked(other, w, dev(t)), y), (F.bf16_grouped_stacked_dgrad(dother, w, dev(t)), dx)):
            assert torch.equal(got[now].view(torch.int16), want[before].view(torch.int16))
    # group g's rows as they are, further ahead: the first group has fewer, and the last rows are no group's
    g = G // 2
    t = [s[0] - s[0] // 3] + s[1:]
    other, _, dother = inputs(G, M, N, K, seed=40)
    a, b, n = sum(s[:g]), sum(t[:g]), s[g]
    other[b:b + n], dother[b:b + n] = x[a:a + n], dy[a:a + n]
    for dtype in (torch.float32, torch.bfloat16):
        got = F.bf16_grouped_stacked_wgrad(dother, other, dev(t), dtype=dtype)
        assert torch.equal(got[g], dw[g].to(dtype))


@pytest.mark.parametrize("G,M,N,K", [(3, 4, 128, 256), (4, 120, 264, 136), (2, 900, 520, 328), (1, 6000, 64, 136)])
def test_gradients_against_differences(F, G, M, N, K):
    """The gradients are those of the forward product: for a loss sum(dY * Y), which is linear in X and in
    W, a step changes it by the step's product with the gradient.  The loss is put together in 64 bits, so
    both sides differ by the roundings of the operators' outputs: 2^-8 of each bf16 value, and the sums' own
    (L + 8) 2^-24 of their magnitudes, weighted as the values are."""
    x, w, dy = inputs(G, M, N, K)
    s = sizes_of(G, M, "skewed")
    used = sum(s)
    sx, sw, _ = inputs(G, M, N, K, seed=9)
    d = dy[:used].double()
    for gradient, step, y, L, bf16 in (
            (F.bf16_grouped_stacked_dgrad(dy, w, dev(s))[:used], sx[:used], F.bf16_grouped_stacked(sx, w, dev(s))[:used], N + K, True),
            (F.bf16_grouped_stacked_wgrad(dy, x, dev(s)), sw, F.bf16_grouped_stacked(x, sw, dev(s))[:used], M + K, False)):
        along = gradient.double() * step.double()
        change = d * y.double()
        size = O.forward((sx if bf16 else x).double(), (w if bf16 else sw).double(), s)[1][:used]
        tol = 2.0 ** -8 * float(change.abs().sum() + (along.abs().sum() if bf16 else 0)) + (L + 16) * 2.0 ** -24 * float((d.abs() * size).sum())
        assert abs(float(along.sum() - change.sum())) <= 1.01 * tol


def test_binding(F):
    x, w, dy = inputs(2, 64, 128, 256)
    s = dev([30, 34])
    ws = torch.empty(0, dtype=torch.uint8, device="cuda")
    assert torch.equal(F.bf16_grouped_stacked_wgrad(dy, x, s, workspace=ws), F.bf16_grouped_stacked_wgrad(dy, x, s))
    assert F.bf16_grouped_stacked_wgrad(dy, x, s).dtype is torch.float32
    assert F.bf16_grouped_stacked_wgrad(dy, x, s, dtype=torch.bfloat16).dtype is torch.bfloat16
    long = inputs(1, 8192, 128, 256)
    for call, text in [
            (lambda: F.bf16_grouped_stacked(x, w.transpose(1, 2), s), "contiguous"),
            (lambda: F.bf16_grouped_stacked(x[:, :128], w, s), "shape|contiguous"),
            (lambda: F.bf16_grouped_stacked(x, w, s.int()), "int64"),
            (lambda: F.bf16_grouped_stacked(x, w, s[:1]), "shape"),
            (lambda: F.bf16_grouped_stacked(x, w, s.cpu()), "on the GPU"),
            (lambda: F.bf16_grouped_stacked(x, w, s, Y=dy.float()), "bfloat16"),
            (lambda: F.bf16_grouped_stacked(x, w, s, Y=dy[:60]), "shape"),
            (lambda: F.bf16_grouped_stacked(dy[:, :124].contiguous(), w[:, :, :124].contiguous(), s), "multiples of 8"),
            (lambda: F.bf16_grouped_stacked_dgrad(x, w, s), "shape"),
            (lambda: F.bf16_grouped_stacked_dgrad(dy, w, s, dX=w[0, :64]), "overlaps"),
            (lambda: F.bf16_grouped_stacked_wgrad(dy, x[:60], s), "shape"),
            (lambda: F.bf16_grouped_stacked_wgrad(dy, x, s, accumulate=True), "dW"),
            (lambda: F.bf16_grouped_stacked_wgrad(dy, x, s, dW=w.clone(), accumulate=True), "fp32"),
            (lambda: F.bf16_grouped_stacked_wgrad(dy, x, s, dW=w.double()), "bfloat16 or float32"),
            (lambda: F.bf16_grouped_stacked_wgrad(long[2], long[0], dev([8192]), workspace=ws), "workspace")]:
        with pytest.raises(ValueError, match=text):
            call()
