"""GPU parity of routing, its plan and its gradient (64-bit oracle).

The choice has to be the oracle's, ties to the lowest index included.  Weights: expf is
off by 2 u, its argument by |x - max| u <= 40 u, the sum of at most 1024 terms by 22 u,
quotient and scale by 2 u: 2^-17 relative covers them.
"""
import numpy as np
import pytest
import torch

from oracle import layer as L
from tests import layer_parity as P

pytestmark = pytest.mark.gpu
REL = 2.0 ** -17


@pytest.fixture(scope="module")
def F():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    import fp8_rowwise_scaled_amd as F
    F.load()
    return F


def check(F, x, k, bias=None, label="", **kw):
    """One call against the oracle: choice, weights and plan."""
    T, E = x.shape
    outs = [P.Guarded((T, k), torch.float32), P.Guarded((T, k), torch.int32), P.Guarded((E,), torch.int64),
            P.Guarded((T, k), torch.int32)]
    r = F.f8f8bf16_route(x.cuda(), k, bias=None if bias is None else bias.cuda(), weights=outs[0].t, ids=outs[1].t,
                         M_sizes=outs[2].t, dst_row=outs[3].t, **kw)
    torch.cuda.synchronize()
    for o in outs:
        o.check(label)
    w, ids = L.route(x.double().numpy(), k, None if bias is None else bias.double().numpy(), **kw)
    got = r.ids.cpu().numpy()
    bad = np.flatnonzero((got != ids).any(1))
    assert bad.size == 0, f"{label}: token {bad[0]} of {bad.size}: {got[bad[0]]} for {ids[bad[0]]}"
    P.assert_close(r.weights, w, REL * np.abs(w) + 1e-37, label + " weights")
    sizes, dst = L.plan(ids, E)
    assert np.array_equal(r.M_sizes.cpu().numpy(), sizes), label
    assert np.array_equal(r.dst_row.cpu().numpy(), dst), label
    return r


SHAPES = [(1, 1, 1), (1, 8, 2), (16, 8, 2), (3, 2, 2), (64, 16, 4), (65, 17, 3), (200, 32, 8), (129, 40, 6), (63, 64, 16),
          (150, 100, 8), (257, 128, 8), (100, 160, 6), (300, 256, 8), (77, 255, 5), (40, 384, 8), (30, 512, 16), (20, 600, 7),
          (15, 1024, 16), (13, 1023, 3)]


@pytest.mark.parametrize("T,E,k", SHAPES)
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("biased", [False, True])
def test_plain_routing(F, T, E, k, score, biased):
    print(f"case route T={T} E={E} k={k} {score} bias={biased}", flush=True)
    rng = np.random.default_rng(T * 1000 + E + k)
    x = torch.from_numpy(rng.normal(0, 2, (T, E)).astype(np.float32))
    if (T + E) % 2:
        x = x.to(torch.bfloat16)
    b = torch.from_numpy(rng.normal(0, 0.1, E).astype(np.float32)) if biased else None
    check(F, x, k, b, score=score, renormalize=bool(k % 2), scale=2.5)
    check(F, x, k, b, score=score, renormalize=not k % 2)


@pytest.mark.parametrize("T,E,n_group,topk_group,k", [(70, 256, 8, 4, 8), (33, 160, 8, 3, 6), (20, 64, 16, 5, 4), (65, 12, 3, 1, 4),
                                                       (40, 16, 16, 2, 2), (25, 96, 2, 2, 16), (10, 1024, 8, 2, 8),
                                                       (12, 600, 4, 2, 5)])
@pytest.mark.parametrize("group_top", [1, 2])
@pytest.mark.parametrize("score,biased", [("softmax", False), ("sigmoid", True), ("softmax", True), ("sigmoid", False)])
def test_groups(F, T, E, n_group, topk_group, k, group_top, score, biased):
    print(f"case groups T={T} E={E} n={n_group} keep={topk_group} k={k} top={group_top} {score} {biased}", flush=True)
    rng = np.random.default_rng(E + n_group * 7 + k)
    x = torch.from_numpy(rng.normal(0, 1.5, (T, E)).astype(np.float32))
    b = torch.from_numpy(rng.normal(0, 0.1, E).astype(np.float32)) if biased else None
    # k may pass what the kept groups hold: the last slots stay empty
    check(F, x, k, b, score=score, n_group=n_group, topk_group=topk_group, group_top=group_top)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E", [8, 60, 256, 320])
def test_ties(F, score, E):
    """Coarse logits make many exact ties, and biases that differ by less than fp32 sees
    in the sum separate some of them."""
    rng = np.random.default_rng(E)
    x = torch.from_numpy(rng.integers(-2, 3, (90, E)).astype(np.float32))
    k = min(8, E)
    check(F, x, k, score=score)
    check(F, x, k, torch.zeros(E), score=score, label="zero bias")
    b = torch.from_numpy((rng.integers(0, 3, E) * 2.0 ** -30).astype(np.float32))
    check(F, x, k, b, score=score, label="tiny bias")
    if E % 4 == 0:
        check(F, x, min(k, E // 4), b, score=score, n_group=4, topk_group=2, group_top=2, label="groups")


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_neighbours_closer_than_fp32(F, score):
    """Scores that fp32 rounds alike (logits one step apart around 8 to 20) in any order."""
    rng = np.random.default_rng(11)
    base = np.float32(rng.uniform(8, 20, (64, 1)))
    steps = rng.permuted(np.tile(np.arange(32), (64, 1)), axis=1).astype(np.float32)
    x = torch.from_numpy((base + steps * np.float32(2.0 ** -19)).astype(np.float32))
    b = torch.from_numpy(rng.choice([0.0, 0.25], 32).astype(np.float32))
    check(F, x, 8, b, score=score)
    check(F, x, 8, b, score=score, n_group=4, topk_group=2, group_top=2)


def test_large_biases_that_cancel_in_a_group(F):
    """One expert of each group is pushed up by 64 and the others down: the groups' sums are
    small while fp32 rounds each key to steps of 2^-17."""
    rng = np.random.default_rng(13)
    x = torch.from_numpy((rng.normal(0, 1, (400, 1)) + rng.normal(0, 2.0 ** -14, (400, 32))).astype(np.float32))
    b = np.full(32, -64.0, np.float32)
    b[rng.integers(0, 8, 4) + 8 * np.arange(4)] = 64.0
    for score in ("softmax", "sigmoid"):
        check(F, x, 4, torch.from_numpy(b), score=score, n_group=4, topk_group=2, group_top=2)
        check(F, x, 4, torch.from_numpy(b), score=score)


def test_masks_and_infinities(F):
    rng = np.random.default_rng(12)
    x = rng.normal(0, 1, (80, 48)).astype(np.float32)
    x[0] = -np.inf                                     # nothing left
    x[1, 3:] = -np.inf                                 # fewer than k left
    x[2, ::2] = np.nan
    x[3, [5, 9]] = np.inf                              # both count as the largest finite value
    x[4] = np.finfo(np.float32).min                    # a mask of the type's lowest value is not a mask
    x[5, :47] = np.finfo(np.float32).min
    x[6, 7] = np.inf
    x[7] = -200.0                                      # sigmoids that fp32 cannot hold
    x[8:40][rng.random((32, 48)) < 0.9] = -np.inf
    x[9, :24], x[9, 24:] = -0.0, 0.0
    t = torch.from_numpy(x)
    b = rng.normal(0, 0.1, 48).astype(np.float32)
    b[10] = -np.inf
    b[20] = np.inf
    b[21] = np.nan
    for score in ("softmax", "sigmoid"):
        for renorm in (True, False):
            kw = dict(score=score, renormalize=renorm)
            check(F, t, 6, **kw)
            check(F, t, 6, torch.from_numpy(b), **kw)
            check(F, t, 6, n_group=8, topk_group=3, group_top=1, **kw)
            check(F, t, 6, torch.from_numpy(b), n_group=8, topk_group=3, group_top=2, **kw)


@pytest.mark.parametrize("T,E,k", [(64, 60, 4), (65, 60, 4), (1000, 60, 4), (16384, 60, 4), (16385, 60, 4), (40000, 60, 4),
                                   (40000, 61, 9), (70000, 256, 16), (3000, 1000, 5)])
def test_many_tokens(F, T, E, k):
    """One to 256 rows of counts, then several passes per workgroup, and more
    pairs per wave of the plan than its registers hold; compared with a sort on the GPU,
    the oracle being slow here."""
    g = torch.Generator(device="cuda").manual_seed(T)
    x = torch.randn(T, E, generator=g, device="cuda")
    r = F.f8f8bf16_route(x, k)
    ids = torch.sort(x, dim=1, descending=True, stable=True).indices[:, :k]
    assert torch.equal(r.ids.long(), ids)
    flat = ids.reshape(-1)
    assert torch.equal(r.M_sizes, (flat[:, None] == torch.arange(E, device="cuda")).sum(0))
    order = torch.sort(flat, stable=True).indices
    assert torch.equal(r.dst_row.view(-1)[order].long(), torch.arange(T * k, device="cuda"))
    assert torch.allclose(r.weights.sum(1), torch.ones(T, device="cuda"), rtol=1e-5)


@pytest.mark.parametrize("T,E,k", [(511, 61, 8), (512, 61, 8), (513, 61, 8), (4096, 8, 1), (4097, 8, 1), (256, 1024, 16), (257, 1024, 16)])
def test_plan_by_one_workgroup_and_by_several(F, T, E, k):
    """Both sides of 4096 pairs, with rows that have fewer experts left than k, or none."""
    g = torch.Generator(device="cuda").manual_seed(T)
    x = torch.randn(T, E, generator=g, device="cuda")
    x[3::7] = -torch.inf
    x[3::14, : max(k // 2, 1)] = 1.0
    r = F.f8f8bf16_route(x, k)
    flat = r.ids.reshape(-1).long()
    left = (x > -torch.inf).sum(1).clamp(max=k)
    assert torch.equal((r.ids >= 0).sum(1), left)
    assert torch.equal(r.M_sizes, (flat[:, None] == torch.arange(E, device="cuda")).sum(0))
    order = torch.sort(torch.where(flat < 0, E, flat), stable=True).indices
    n = int(left.sum())
    want = torch.full((T * k,), -1, dtype=torch.int64, device="cuda")
    want[order[:n]] = torch.arange(n, device="cuda")
    assert torch.equal(r.dst_row.view(-1).long(), want)


@pytest.mark.parametrize("E", [8, 60, 100, 128, 200, 256, 300, 512, 700])
@pytest.mark.parametrize("score,renormalize", [("softmax", False), ("softmax", True), ("sigmoid", False)])
def test_rows_do_not_depend_on_the_batch(F, E, score, renormalize):
    """The same bits, however many tokens a call has and with or without the plan."""
    g = torch.Generator(device="cuda").manual_seed(E)
    x = torch.randn(20000, E, generator=g, device="cuda")
    b = 0.1 * torch.randn(E, generator=g, device="cuda")
    kw = dict(bias=b, score=score, renormalize=renormalize, n_group=4, topk_group=3, group_top=2)
    all_of = F.f8f8bf16_route(x, 5, **kw)
    for start, n in [(0, 1), (3, 6), (9, 17), (64, 64), (100, 200), (300, 1000), (2000, 4096), (10000, 5000)]:
        for plan in (True, False):
            r = F.f8f8bf16_route(x[start : start + n], 5, plan=plan, **kw)
            assert torch.equal(r.ids, all_of.ids[start : start + n]), (start, n, plan)
            assert torch.equal(r.weights, all_of.weights[start : start + n]), (start, n, plan)


def test_no_tokens_and_no_plan(F):
    r = F.f8f8bf16_route(torch.empty((0, 8), device="cuda"), 2)
    assert torch.equal(r.M_sizes, torch.zeros(8, dtype=torch.int64, device="cuda")) and r.ids.shape == (0, 2)
    x = torch.randn(300, 32, device="cuda")
    a, b = F.f8f8bf16_route(x, 4), F.f8f8bf16_route(x, 4, plan=False)
    assert b.M_sizes is None and b.dst_row is None and torch.equal(a.ids, b.ids) and torch.equal(a.weights, b.weights)


@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (5, 8, 2), (130, 17, 3), (64, 128, 8), (33, 250, 16), (20, 1024, 16), (3, 1001, 4)])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renormalize", [True, False])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_backward(F, T, E, k, score, renormalize, dtype):
    print(f"case route backward T={T} E={E} k={k} {score} {renormalize} {dtype}", flush=True)
    rng = np.random.default_rng(T + E * 3 + k)
    x = torch.from_numpy(rng.normal(0, 2, (T, E)).astype(np.float32)).to(dtype)
    _, ids = L.route(x.double().numpy(), k, score=score)
    if T > 2:
        ids[1, k // 2:] = -1
        ids[2, 0] = E + 5
    dw = torch.from_numpy(rng.normal(0, 1, (T, k)).astype(np.float32))
    out = P.Guarded((T, E), dtype)
    F.f8f8bf16_route_backward(x.cuda(), torch.from_numpy(ids.astype(np.int32)).cuda(), dw.cuda(), score=score,
                              renormalize=renormalize, scale=1.5, dlogits=out.t)
    torch.cuda.synchronize()
    out.check()
    want, size = L.route_backward(x.double().numpy(), ids, dw.double().numpy(), score, renormalize, 1.5)
    P.assert_close(out.t, want, (P.BF16 if dtype == torch.bfloat16 else 0) * np.abs(want) + REL * size + 1e-37, "dlogits")


def test_backward_with_masked_logits(F):
    x = torch.zeros((3, 8))
    x[0, 2:] = -float("inf")
    x[1] = -float("inf")
    ids = torch.tensor([[0, 1, -1], [-1, -1, -1], [0, 1, 2]], dtype=torch.int32)
    for score in ("softmax", "sigmoid"):
        for renorm in (True, False):
            d = F.f8f8bf16_route_backward(x.cuda(), ids.cuda(), torch.ones(3, 3, device="cuda"), score=score, renormalize=renorm)
            want, size = L.route_backward(x.double().numpy(), ids.numpy(), np.ones((3, 3)), score, renorm)
            P.assert_close(d, want, REL * size + 1e-37)


def test_offsets_past_31_bits(F):
    """Logits past element 2^31, more tokens per workgroup than one pass, and a plan of 18
    million pairs."""
    T, E, k = 9_000_000, 256, 2
    g = torch.Generator(device="cuda").manual_seed(2)
    x = torch.empty((T, E), dtype=torch.bfloat16, device="cuda")
    x.normal_(generator=g)
    r = F.f8f8bf16_route(x, k)
    tail = F.f8f8bf16_route(x[-100:].contiguous(), k)
    assert torch.equal(r.ids[-100:], tail.ids) and torch.equal(r.weights[-100:], tail.weights)
    flat = r.ids.view(-1)
    assert torch.equal(r.M_sizes, torch.bincount(flat, minlength=E))
    starts = torch.cumsum(r.M_sizes, 0) - r.M_sizes
    dst = r.dst_row.view(-1).long()
    place = torch.zeros(T * k, dtype=torch.bool, device="cuda")
    place[dst] = True
    assert bool(place.all())                                  # a permutation
    order = torch.sort(flat.to(torch.int16), stable=True).indices
    assert torch.equal(dst[order], torch.arange(T * k, device="cuda"))
    assert bool((dst >= starts[flat.long()]).all())
    dw = torch.rand((T, k), device="cuda", generator=g)
    d = F.f8f8bf16_route_backward(x, r.ids, dw)
    e = F.f8f8bf16_route_backward(x[-100:].contiguous(), tail.ids, dw[-100:].contiguous())
    assert torch.equal(d[-100:], e)
