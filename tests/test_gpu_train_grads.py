"""GPU parity of the gradients' norm and clipping with the 64-bit oracle.

Squares and their sum are in fp64 (2^-53 each, not seen next to what follows).  The norm is rounded to fp32
(2^-24); the factor is rounded to fp32 and multiplies in fp32: two half steps of 2^-24; a bf16 result
rounds once more, 2^-8.  Results below fp32's normal range are off by half of its smallest step."""
import math

import pytest
import torch

from oracle import train as O

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


@pytest.fixture(scope="module")
def F():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    import fp8_rowwise_scaled_amd as F
    F.load()
    return F


def make(sizes, seed=0, sigma=1e-3):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return [(torch.randn(n, generator=g, device="cuda") * sigma).to(torch.bfloat16 if i % 3 == 1 else torch.float32) for i, n in enumerate(sizes)]


def check(F, grads, max_norm, eps=1e-6, into=False, **kw):
    norm, factor, want = O.clip(grads, max_norm, eps)
    outs = [torch.full_like(g, 7.0) for g in grads] if into else None
    before = [g.clone() for g in grads]
    got = F.f8f8bf16_grad_clip(grads, max_norm, eps, outs=outs, **kw)
    torch.cuda.synchronize()
    assert got.shape == (1,) and got.dtype is torch.float32 and got.is_cuda
    if norm > 2.0 ** 128:                                # rounds to fp32's infinity; the factor does not go by that
        assert math.isinf(float(got))
    else:
        assert abs(float(got) - norm) <= 1.01 * U * norm + 2.0 ** -150
    if into:
        assert all(torch.equal(a, b) for a, b in zip(grads, before))
    for i, (g, w) in enumerate(zip(outs if into else grads, want)):
        tol = 2.02 * U * w.abs() + 2.0 ** -149 + (2.0 ** -8 * 1.001 * w.abs() + 2.0 ** -133 if g.dtype is torch.bfloat16 else 0)
        assert bool(((g.double() - w).abs() <= tol).all()), f"tensor {i}"
        if factor == 1.0:
            assert torch.equal(g, before[i])
    return float(got)


SIZES = [[1], [7, 1, 3], [4096], [100000, 5, 0, 8193], [16384 * 3 + 5, 4095, 4097], [3, 0, 0, 2], [1 << 20, 1 << 21, 12345, 77], list(range(1, 250))]


@pytest.mark.parametrize("sizes", SIZES, ids=lambda s: f"{len(s)}x{max(s)}")
@pytest.mark.parametrize("into", [False, True])
def test_norm_and_clip(F, sizes, into):
    print(f"case clip {len(sizes)} tensors, {sum(sizes)} values, into={into}", flush=True)
    norm = math.sqrt(sum(sizes)) * 1e-3
    for bound in (0.3 * norm, 30 * norm, 0.0, float("inf")):
        check(F, make(sizes), bound, into=into)
    check(F, make(sizes), norm, eps=0.5 * norm, into=into)


def test_square_sum(F):
    grads = make([1000, 3, 70000, 0, 16384])
    want = math.fsum(float(v) ** 2 for g in grads for v in g.double().flatten().tolist())
    got = F.f8f8bf16_grad_square_sum(grads)
    assert got.dtype is torch.float64 and abs(float(got) - want) <= 1e-12 * want
    # two ranks' sums added up, each clipping its own tensors by the common norm
    other = make([500, 2000], seed=3)
    total = got + F.f8f8bf16_grad_square_sum(other)
    norm = math.sqrt(float(total))
    scaled = [g.clone() for g in other]
    n = F.f8f8bf16_grad_clip(scaled, 0.5 * norm, eps=0.0, square_sum=total)
    assert abs(float(n) - norm) <= 1.01 * U * norm
    for a, b in zip(scaled, other):
        assert bool(((a.double() - 0.5 * b.double()).abs() <= 2.02 * U * b.double().abs() + (2.0 ** -8 * b.double().abs() if b.dtype is torch.bfloat16 else 0)).all())


def test_no_tensors(F):
    assert float(F.f8f8bf16_grad_square_sum([])) == 0.0 and float(F.f8f8bf16_grad_clip([], 1.0)) == 0.0
    assert float(F.f8f8bf16_grad_clip((torch.zeros(0, device="cuda"),), 1.0)) == 0.0
    assert float(F.f8f8bf16_grad_square_sum([torch.zeros(0, device="cuda")] * 3)) == 0.0


@pytest.mark.parametrize("value", [1e-30, 1e30, 3e38, 1e-44])
def test_squares_that_fp32_does_not_hold(F, value):
    grads = [torch.full((5000,), value, device="cuda"), torch.full((300,), value, device="cuda").to(torch.bfloat16)]
    check(F, [g.clone() for g in grads], 0.5 * math.sqrt(5300) * value, eps=0.0)


def test_infinite_and_nan_gradients(F):
    def grads(bad):
        g = make([5000, 3000])
        g[0][17] = bad
        return g
    a = grads(float("inf"))
    assert math.isinf(float(F.f8f8bf16_grad_clip(a, 1.0)))
    assert bool(a[0][17].isnan()) and float(a[0].nan_to_num(0).abs().max()) == 0.0 and not a[1].any()
    a = grads(float("nan"))
    assert math.isnan(float(F.f8f8bf16_grad_clip(a, 1.0))) and all(bool(g.isnan().all()) for g in a)


@pytest.mark.parametrize("into", [False, True])
@pytest.mark.parametrize("bad", [float("inf"), -float("inf"), float("nan")])
def test_an_infinite_bound_leaves_every_gradient(F, bad, into):
    """The norm alone: also where it is infinite or NaN, no value changes, in place or on its way into outs."""
    g = make([5000, 3000, 20000])
    g[0][17] = bad
    before = [t.clone() for t in g]
    outs = [torch.full_like(t, 7.0) for t in g] if into else None
    norm = float(F.f8f8bf16_grad_clip(g, float("inf"), outs=outs))
    assert math.isnan(norm) if math.isnan(bad) else norm == math.inf
    for a, b in zip(outs if into else g, before):
        keep = ~b.isnan()
        assert torch.equal(a[keep], b[keep]) and bool(a[~keep].isnan().all())
    assert float(F.f8f8bf16_grad_clip(g, float("inf"), square_sum=torch.full((1,), math.inf, dtype=torch.float64, device="cuda"))) == math.inf
    assert torch.equal(g[1], before[1]) and torch.equal(g[2], before[2])


@pytest.mark.parametrize("into", [False, True])
def test_zeros_stay_zeros_without_eps(F, into):
    """The factor's denominator is 0 there: nothing to scale down, whatever the bound."""
    for bound in (0.0, 1.0, float("inf")):
        g = [torch.zeros(5000, device="cuda"), torch.zeros(3000, dtype=torch.bfloat16, device="cuda")]
        outs = [torch.full_like(t, 7.0) for t in g] if into else None
        assert float(F.f8f8bf16_grad_clip(g, bound, eps=0.0, outs=outs)) == 0.0
        assert not any(bool((t != 0).any()) for t in (outs or g))


@pytest.mark.parametrize("offset", range(8))
def test_views_at_any_alignment(F, offset):
    """Tensors one after another in a flat buffer, in place and into a buffer aligned otherwise; what lies around them stays."""
    for dtype in (torch.float32, torch.bfloat16):
        flat = (torch.randn(60000, device="cuda") * 1e-2).to(dtype)
        sizes = [3, 16389, 1, 40000 - offset]
        parts = list(flat[offset:offset + sum(sizes)].split(sizes))
        keep = flat.clone()
        other = torch.full((60000,), 5.0, device="cuda").to(dtype)
        outs = list(other[1:1 + sum(sizes)].split(sizes))
        norm, factor, want = O.clip(parts, 0.7, 0.0)
        assert factor < 1
        for o in (outs, None):
            F.f8f8bf16_grad_clip(parts, 0.7, 0.0, outs=o)
            torch.cuda.synchronize()
            for g, w in zip(o or parts, want):
                tol = 2.02 * U * w.abs() + (2.0 ** -8 * 1.001 * w.abs() if dtype is torch.bfloat16 else 0)
                assert bool(((g.double() - w).abs() <= tol).all())
            if o:
                assert torch.equal(flat, keep)
                assert bool((other[:1] == 5).all()) and bool((other[1 + sum(sizes):] == 5).all())
        assert torch.equal(flat[:offset], keep[:offset]) and torch.equal(flat[offset + sum(sizes):], keep[offset + sum(sizes):])


def test_strided_but_dense(F):
    base = torch.randn(64, 48, device="cuda")
    norm, _, want = O.clip([base], 0.0, 0.0)
    want = base.double() * 0.5
    t = base.t()
    n = F.f8f8bf16_grad_clip([t], norm * 0.5, eps=0.0)
    assert abs(float(n) - norm) <= 1.01 * U * norm
    assert bool(((base.double() - want).abs() <= 2.02 * U * want.abs()).all())
    for call, text in [
            (lambda: F.f8f8bf16_grad_clip([base[:, ::2]], 1.0), "dense"),
            (lambda: F.f8f8bf16_grad_clip([base[:1].expand(4, 48)], 1.0), "dense"),
            (lambda: F.f8f8bf16_grad_clip([t], 1.0, outs=[torch.empty(48, 64, device="cuda")]), "strides"),
            (lambda: F.f8f8bf16_grad_clip([base], 1.0, outs=[]), "outs"),
            (lambda: F.f8f8bf16_grad_clip([base, base], 1.0), "overlaps"),
            (lambda: F.f8f8bf16_grad_clip([base[:40], base[30:]], 1.0), "overlaps"),
            (lambda: F.f8f8bf16_grad_clip([base], 1.0, square_sum=torch.zeros(1, device="cuda")), "float64"),
            (lambda: F.f8f8bf16_grad_clip([base, base.cpu()], 1.0), "on the GPU"),
            (lambda: F.f8f8bf16_grad_clip([base], -1.0), "max_norm"),
            (lambda: F.f8f8bf16_grad_clip([base], 1.0, workspace=torch.empty(8, device="cuda")), "workspace")]:
        with pytest.raises(ValueError, match=text):
            call()
    # read only, the same tensor may come twice
    assert abs(float(F.f8f8bf16_grad_square_sum([base, base])) - 2 * float(base.double().square().sum())) < 1e-9 * float(base.double().square().sum())


def test_more_than_31_bits_of_values(F):
    n = (1 << 31) + 12345
    g = torch.zeros(n, dtype=torch.bfloat16, device="cuda")
    g[-1], g[5] = 3.0, 4.0
    assert float(F.f8f8bf16_grad_clip([g], 1.0, eps=0.0)) == 5.0
    assert abs(float(g[-1]) - 0.6) < 0.002 and abs(float(g[5]) - 0.8) < 0.003 and int(g.count_nonzero()) == 2


def test_a_list_that_loses_its_tensors_during_the_call(F):
    """A bound that is turned into a number by the caller's code, which empties the list: the call has its tensors all the same."""
    class Bound:
        def __init__(self, *lists):
            self.lists = lists

        def __float__(self):
            for x in self.lists:
                x.clear()
            return 0.5 * norm
    kept = make([4096, 12345])
    norm = math.sqrt(sum(float(g.double().square().sum()) for g in kept))
    want = O.clip(kept, 0.5 * norm, 0.0)[2]
    views = [torch.empty_like(g) for g in kept]
    grads, outs = [g.clone() for g in kept], list(views)
    got = F.f8f8bf16_grad_clip(grads, Bound(grads), eps=0.0, outs=outs)
    assert grads == [] and abs(float(got) - norm) <= 1.01 * U * norm
    grads = [g.clone() for g in kept]
    held = list(grads)
    F.f8f8bf16_grad_clip(grads, Bound(grads), eps=0.0)
    for a, b, w in zip(views, held, want):
        assert torch.equal(a, b)
        assert bool(((a.double() - w).abs() <= 2.02 * U * w.abs() + (2.0 ** -8 * 1.001 * w.abs() if a.dtype is torch.bfloat16 else 0)).all())


def test_results_do_not_depend_on_the_run(F):
    grads = make([1 << 22, 12345, 1 << 20])
    first = [float(F.f8f8bf16_grad_square_sum(grads)) for _ in range(4)]
    assert len(set(first)) == 1
    big = make(list(range(2000, 2300)))
    assert len({float(F.f8f8bf16_grad_square_sum(big)) for _ in range(4)}) == 1
