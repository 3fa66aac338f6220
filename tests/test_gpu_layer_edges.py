"""GPU tests of the layer operators at the edges of their ranges: values near the ends of
fp32, rows and places that hold nothing, more work than one pass of a grid, and rows of
the router that leave its usual path."""
import numpy as np
import pytest
import torch

from oracle import layer as L
from tests import layer_parity as P
from tests.test_gpu_layer_route import check

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def F():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    import fp8_rowwise_scaled_amd as F
    F.load()
    return F


LOWEST = float(np.finfo(np.float32).min)


@pytest.mark.parametrize("T,per", [(40, 4), (40, 40), (4200, 40)])     # 16 lanes per token, 64, 16 with several keys each
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_group_sums_past_fp32(F, T, per, score):
    """Sums of two keys that fp32 cannot hold: a bias of the type's lowest value takes no group
    out, and sums above the largest value keep their order."""
    print(f"case group sums T={T} per={per} {score}", flush=True)
    rng = np.random.default_rng(per)
    x = torch.from_numpy(rng.normal(0, 1, (T, 4 * per)).astype(np.float32))

    def bias(**of):
        b = rng.normal(0, 0.1, (4, per)).astype(np.float32)
        for g, v in of.items():
            b[int(g[1:]), :len(v)] = v
        return torch.from_numpy(b.reshape(-1))
    low = bias(g0=[LOWEST] * per, g2=[LOWEST] * per)
    for keep in (1, 3, 4):
        check(F, x, 12, low, score=score, n_group=4, topk_group=keep, group_top=2, label=f"lowest, keep {keep}")
    high = bias(g1=[3e38, 0.5e38], g2=[3e38, 3e38], g3=[0.9e38, 3e38])
    for keep in (1, 2, 3):
        check(F, x, 4, high, score=score, n_group=4, topk_group=keep, group_top=2, label=f"large, keep {keep}")
    check(F, x, 4, bias(g0=[-3e38] * per, g1=[-2e38] * per, g2=[-2.5e38] * per, g3=[-np.inf] * per), score=score, n_group=4,
          topk_group=2, group_top=2, label="negative")
    check(F, x, 4, bias(g1=[np.inf, np.inf], g3=[np.inf, np.inf]), score=score, n_group=4, topk_group=1, group_top=2,
          label="infinite")


@pytest.mark.parametrize("k", [1, 2, 3])
@pytest.mark.parametrize("N", [264, 2056, 4104, 8200])
def test_left_out_places_have_no_weight_gradient(F, N, k):
    """... whatever their token's gradient holds."""
    print(f"case left out N={N} k={k}", flush=True)
    T, R = 24, 24 * k
    g = torch.Generator(device="cuda").manual_seed(N + k)
    dout = torch.randn(T, N, generator=g, device="cuda").to(torch.bfloat16)
    dout[3, N // 2], dout[4, 5], dout[5] = float("nan"), float("inf"), -float("inf")
    y = torch.randn(R, N, generator=g, device="cuda").to(torch.bfloat16)
    dst = torch.randperm(T * k, generator=g, device="cuda").to(torch.int32).view(T, k)
    out = torch.zeros((T, k), dtype=torch.bool, device="cuda")
    out[::2, k - 1], out[3:6, 0] = True, True
    dst[out] = torch.where(torch.arange(int(out.sum()), device="cuda") % 2 == 0, -1, R).to(torch.int32)
    _, dw = F.f8f8bf16_moe_combine_backward(dout, dst, torch.ones(T, k, device="cuda"), y)
    assert torch.all(dw[out] == 0), dw[out]
    good = ~out
    good[3:6] = False
    assert torch.all(dw[good] != 0) and torch.all(torch.isfinite(dw[good]))


@pytest.mark.parametrize("K", [256, 1024, 2048, 4096, 7168, 8192, 16384, 20480])
@pytest.mark.parametrize("block", [0, 128])
@pytest.mark.parametrize("eps", [0.0, 1e-38])
def test_norm_of_rows_whose_squares_leave_fp32(F, K, block, eps):
    """Rows down to 2^-90: their squares are below what fp32 holds, their norm is not.  A row of
    zeros has rstd 0 without eps, so that neither it nor its gradient holds a NaN."""
    print(f"case small rows K={K} block={block} eps={eps}", flush=True)
    rng = np.random.default_rng(K)
    powers = [0, -40, -48, -50, -60, -64, -70, -80, -90]
    x = rng.normal(0, 1, (len(powers) + 1, K)) * 2.0 ** np.array(powers + [0], np.float64)[:, None]
    x[-1] = 0.0
    x = P.to_bf16(x)
    res = torch.zeros_like(x)
    w = torch.from_numpy(rng.normal(1, 0.3, K).astype(np.float32))
    for residual in (None, res.cuda()):
        # in place: the branch may not read a residual that has been overwritten
        out = F.f8f8bf16_rmsnorm_quantize(x.cuda(), w.cuda(), eps, residual=residual, residual_out=residual, block=block,
                                          want_y=True, want_rstd=True)
        X, W, E = P.f64(x), P.f64(w), np.float64(np.float32(eps))
        with np.errstate(divide="ignore", invalid="ignore"):
            h, y, rstd = L.rmsnorm(X, None, W, E)
        if eps == 0.0:
            y[-1], rstd[-1] = 0.0, 0.0
        P.assert_close(out.rstd, rstd, 2.0 ** -18 * rstd, "rstd")
        P.assert_close(out.Y, y, (P.BF16 + 2.0 ** -18) * np.abs(y) + 1e-40, "Y")
        hw = L.block_amax(X * W, block)
        scale = np.where(hw > 0, np.maximum(hw, 2.0 ** -100) / 448 * (rstd if not block else rstd[:, None]), 1.0)
        P.assert_close(out.x_scale, scale, 2.0 ** -18 * scale, "x_scale")
        P.assert_codes(out.XQ, X * W / L.spread(L.scale_of(hw), K), 2.0 ** -21, "codes")
    dy = P.to_bf16(rng.normal(0, 1, x.shape) * 1e-2)
    dx, dw = F.f8f8bf16_rmsnorm_backward(dy.cuda(), x.cuda(), w.cuda(), out.rstd, res.cuda())
    R, DY = P.f64(out.rstd), P.f64(dy)
    want, want_w = L.rmsnorm_backward(DY, X, W, R, None)
    xhat = X * R[:, None]
    size = R[:, None] * (np.abs(DY * W) + np.abs(xhat) * np.abs(DY * W * xhat).mean(1, keepdims=True))
    P.assert_close(dx, want, P.BF16 * np.abs(want) + 2.0 ** -18 * size + 1e-40, "dX")
    P.assert_close(dw, want_w, (x.shape[0] + 48) * P.U * np.abs(DY * xhat).sum(0) + 1e-30, "dweight")


def test_integers_are_not_cut(F):
    """Integers past 32 bits are refused, not taken for their low half."""
    x = torch.randn(8, 32, device="cuda")
    dst = torch.zeros((8, 1), dtype=torch.int32, device="cuda")
    q, s = torch.zeros((8, 32), dtype=torch.uint8, device="cuda"), torch.ones(8, device="cuda")
    for call, text in [(lambda: F.f8f8bf16_route(x, 2, n_group=4, topk_group=2, group_top=2 ** 32 + 2), "group_top"),
                       (lambda: F.f8f8bf16_route(x, 2, group_top=1 - 2 ** 32), "group_top"),
                       (lambda: F.f8f8bf16_rmsnorm_quantize(x.to(torch.bfloat16), s.new_ones(32), block=2 ** 32), "block"),
                       (lambda: F.f8f8bf16_moe_dispatch(q, s, dst, rows=2 ** 40), "too large"),
                       (lambda: F.f8f8bf16_moe_combine_backward(x.to(torch.bfloat16), dst, rows=2 ** 40), "too large")]:
        with pytest.raises(ValueError, match=text):
            call()


@pytest.mark.parametrize("T,k,K,cols", [(5, 8, 64, 3), (9, 64, 512, 65), (3, 40, 304, 300), (4, 33, 4096, 256), (2, 3, 8192, 500)])
def test_dispatch_of_any_number_of_scales(F, T, k, K, cols):
    """Fewer scales than a wave has lanes, more than a workgroup, and places in lanes without one."""
    print(f"case dispatch scales T={T} k={k} K={K} cols={cols}", flush=True)
    rng = np.random.default_rng(T + cols)
    R = T * k + 1
    dst = rng.permutation(R)[:T * k].reshape(T, k)
    dst[0, k - 1] = -1
    q, s = rng.integers(0, 256, (T, K), dtype=np.uint8), rng.random((T, cols)).astype(np.float32)
    oq, os_ = P.Guarded((R, K), torch.uint8), P.Guarded((R, cols), torch.float32)
    F.f8f8bf16_moe_dispatch(torch.from_numpy(q).cuda(), torch.from_numpy(s).cuda(), torch.from_numpy(dst.astype(np.int32)).cuda(),
                            rows=R, XQs=oq.t, xs_out=os_.t)
    torch.cuda.synchronize()
    oq.check()
    os_.check()
    for got, rows in ((oq, q), (os_, s)):
        want, written = L.dispatch(rows, dst, R)
        assert np.array_equal(got.t.cpu().numpy()[written], want[written])
        assert np.all(got.untouched(~written))


@pytest.mark.parametrize("T", [90, 4200])                              # 64 and 16 lanes per token
@pytest.mark.parametrize("E", [256, 344])
@pytest.mark.parametrize("kind", ["equal", "padded", "random"])
@pytest.mark.parametrize("score,biased,groups", [("softmax", False, False), ("softmax", True, False), ("sigmoid", True, True),
                                                 ("sigmoid", False, True)])
def test_rows_with_many_candidates(F, T, E, kind, score, biased, groups):
    """More keys than the list of candidates holds: rows of equal logits (all, or every fourth as
    padding leaves them) and k = 16; with and without sums that fp32 cannot tell apart."""
    print(f"case candidates T={T} E={E} {kind} {score} bias={biased} groups={groups}", flush=True)
    rng = np.random.default_rng(T + E)
    x = rng.normal(0, 1, (T, E)).astype(np.float32)
    if kind == "equal":
        x[:] = 0.0
    elif kind == "padded":
        x[3::4] = 0.25
    b = (rng.integers(0, 3, E) * 2.0 ** -30).astype(np.float32) if biased else None
    kw = dict(n_group=8, topk_group=4, group_top=2) if groups else {}
    check(F, torch.from_numpy(x), 16 if kind == "random" else 8, None if b is None else torch.from_numpy(b), score=score, **kw)


def test_weights_of_softmax_with_a_bias_and_bf16_sigmoid(F):
    """What crosses to fp64 most often: keys of many small shares, and bf16 logits that tie."""
    rng = np.random.default_rng(31)
    x = torch.from_numpy(rng.normal(0, 0.5, (4200, 256)).astype(np.float32))
    b = torch.from_numpy(rng.normal(0, 1e-3, 256).astype(np.float32))
    check(F, x, 8, b, score="softmax")
    check(F, x.to(torch.bfloat16), 8, torch.zeros(256), score="sigmoid")


def places(T, k, seed):
    """A permutation of the T k rows, a tenth of the places left out."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    dst = torch.randperm(T * k, generator=g, device="cuda").to(torch.int32).view(T, k)
    dst[torch.rand((T, k), generator=g, device="cuda") < 0.1] = -1
    return g, dst


@pytest.mark.parametrize("T,k,N", [(1_100_000, 1, 8), (1_100_000, 1, 264), (700_000, 3, 16), (1_100_000, 2, 40)])
def test_exchange_of_more_tokens_than_a_grid_has_workgroups(F, T, k, N):
    """A workgroup takes several tokens: 2^20 of them are the most that one launch has."""
    print(f"case exchange T={T} k={k} N={N}", flush=True)
    g, dst = places(T, k, T + N)
    y = torch.randn(T * k, N, generator=g, device="cuda").to(torch.bfloat16)
    # small whole weights and gradients: sums and products are exact in fp32, whatever their order
    w = torch.randint(-4, 5, (T, k), generator=g, device="cuda").float()
    dout = torch.randint(-2, 3, (T, N), generator=g, device="cuda").to(torch.bfloat16)
    y = (y * 4).round() / 4
    here = dst >= 0
    at = dst.long().clamp(min=0)
    rows = torch.where(here[:, :, None], y[at].float(), 0.0)
    out = F.f8f8bf16_moe_combine(y, dst, w)
    assert torch.equal(out, (rows * w[:, :, None]).sum(1).to(torch.bfloat16))
    mark = torch.full_like(y, 7.0)
    dy, dw = F.f8f8bf16_moe_combine_backward(dout, dst, w, y, dY=mark)
    assert torch.equal(dw, (rows * dout.float()[:, None]).sum(2))
    want = torch.full_like(y, 7.0)
    want[at[here]] = (dout.float()[:, None] * w[:, :, None]).to(torch.bfloat16)[here]
    assert torch.equal(dy, want)


def test_dispatch_of_more_tokens_than_a_grid_has_workgroups(F):
    T, k, K = 1_100_000, 2, 16
    g, dst = places(T, k, 5)
    q = torch.randint(0, 256, (T, K), dtype=torch.uint8, generator=g, device="cuda")
    s = torch.rand(T, generator=g, device="cuda")
    out, scales = torch.full((T * k, K), 9, dtype=torch.uint8, device="cuda"), torch.full((T * k,), 9.0, device="cuda")
    want, want_s = out.clone(), scales.clone()
    F.f8f8bf16_moe_dispatch(q, s, dst, XQs=out, xs_out=scales)
    here = dst >= 0
    token = torch.arange(T, device="cuda")[:, None].expand(T, k)[here]
    want[dst[here].long()], want_s[dst[here].long()] = q[token], s[token]
    assert torch.equal(out, want) and torch.equal(scales, want_s)


def test_activation_of_more_rows_than_a_grid_has_workgroups(F):
    """... compared with the same rows in smaller calls."""
    rows, I = 4_300_000, 8
    g = torch.Generator(device="cuda").manual_seed(6)
    h = torch.randn(rows, 2 * I, generator=g, device="cuda").to(torch.bfloat16)
    da = torch.randn(rows, I, generator=g, device="cuda").to(torch.bfloat16)
    a = F.f8f8bf16_silu_mul_quantize(h, checkpoint=True)
    d = F.f8f8bf16_silu_mul_backward(da, a.HQ, a.h_scale)
    for start in (0, 262_144, 2_000_000, 4_194_300, 4_250_000):
        part = slice(start, start + 50_000)
        b = F.f8f8bf16_silu_mul_quantize(h[part], checkpoint=True)
        assert all(torch.equal(x[part], y) for x, y in zip(a, b))
        assert torch.equal(d[part], F.f8f8bf16_silu_mul_backward(da[part], b.HQ, b.h_scale))


@pytest.mark.parametrize("rows,K", [(70_000, 1032), (300_000, 264), (70_000, 2056)])
@pytest.mark.parametrize("block", [0, 128])
def test_norm_of_more_rows_than_a_grid_has_teams(F, rows, K, block):
    """The sums of a team's second row use the other half of its exchange buffer."""
    K = K // 128 * 128 if block else K
    print(f"case norm rows={rows} K={K} block={block}", flush=True)
    g = torch.Generator(device="cuda").manual_seed(rows)
    x = torch.randn(rows, K, generator=g, device="cuda").to(torch.bfloat16)
    w = torch.rand(K, generator=g, device="cuda") + 0.5
    a = F.f8f8bf16_rmsnorm_quantize(x, w, block=block, want_rstd=True)
    for start in (0, 60_000, 65_530, rows - 4000):
        part = slice(start, start + 4000)
        b = F.f8f8bf16_rmsnorm_quantize(x[part], w, block=block, want_rstd=True)
        assert torch.equal(a.XQ[part], b.XQ) and torch.equal(a.x_scale[part], b.x_scale) and torch.equal(a.rstd[part], b.rstd)


@pytest.mark.parametrize("T,E", [(90, 64), (90, 256), (4200, 256)])
@pytest.mark.parametrize("zero_bias", [False, True])
@pytest.mark.parametrize("group_top", [0, 1, 2])
def test_scores_far_below_the_largest(F, T, E, zero_bias, group_top):
    """Experts and groups are told apart by scores far below the row's largest, and by how far
    sigmoids are from 1: exact arithmetic does, and fp64 where the scores are small."""
    print(f"case small scores T={T} E={E} zero bias={zero_bias} group_top={group_top}", flush=True)
    rng = np.random.default_rng(E + T)
    b = torch.zeros(E) if zero_bias else None
    kw = dict(n_group=8, topk_group=4, group_top=group_top) if group_top else {}
    peaked = rng.normal(0, 12, (T, E))
    peaked[::3, rng.integers(0, E)] += 60.0
    check(F, torch.from_numpy(peaked.astype(np.float32)), 8, b, score="softmax", label="peaked", **kw)
    # shares below fp32's range: the plain weights are 0 there, the choice is not open
    far = rng.normal(-60, 10, (T, E))
    far[:, 3] = 90.0
    check(F, torch.from_numpy(far.astype(np.float32)), 8, b, score="softmax", label="far", **kw)
    check(F, torch.from_numpy(rng.normal(-45, 4, (T, E)).astype(np.float32)), 8, b, score="sigmoid", label="low", **kw)
    near_one = rng.uniform(14, 20, (T, E)).astype(np.float32)
    check(F, torch.from_numpy(near_one), 8, b, score="sigmoid", label="near one", **kw)


def test_tensors_without_memory_are_refused(F):
    """A tracer's stand-in for a GPU tensor throws when it is asked for its address: a Python error,
    raised with the interpreter's lock held."""
    from torch._subclasses.fake_tensor import FakeTensorMode
    x = torch.randn(8, 32, device="cuda")
    F.f8f8bf16_route(x, 2)
    with FakeTensorMode() as mode:
        fake = mode.from_tensor(x)
        for _ in range(3):
            with pytest.raises(Exception):
                F.f8f8bf16_route(fake, 2)
    r = F.f8f8bf16_route(x, 2)
    assert torch.equal(r.ids.long(), torch.sort(x, dim=1, descending=True, stable=True).indices[:, :2])


FIRST_CALL = """
import torch
from torch._subclasses.fake_tensor import FakeTensorMode
import fp8_rowwise_scaled_amd as F
x = torch.randn(8, 32, device="cuda")
with FakeTensorMode() as mode:
    fake = mode.from_tensor(x)
    try:
        F.f8f8bf16_route(fake, 2)
    except Exception as e:
        print("refused:", e)
r = F.f8f8bf16_route(x, 2)
assert torch.equal(r.ids.long(), torch.sort(x, dim=1, descending=True, stable=True).indices[:, :2])
print("right")
"""


def test_a_first_call_under_a_tracer_leaves_no_trace():
    """The GPU allocator that the binding keeps is torch's, whatever mode the first call ran in."""
    import os
    import subprocess
    import sys
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", FIRST_CALL], cwd=root, capture_output=True, text=True, timeout=100)
    assert r.returncode == 0 and "refused" in r.stdout and r.stdout.strip().endswith("right"), r.stdout + r.stderr[-2000:]


@pytest.mark.parametrize("block", [0, 128])
def test_activations_of_gates_far_below_zero(F, block):
    """What the header says of them: codes within (|g| + 4) 2^-22 and half a step, scales too."""
    rng = np.random.default_rng(41)
    tops = np.arange(0, -86, -5)
    gate = tops[:, None] - rng.uniform(0, 1, (len(tops), 256))
    up = rng.normal(0, 1, gate.shape) * 2.0 ** 60
    h = P.to_bf16(np.concatenate([gate, up], axis=1))
    out = F.f8f8bf16_silu_mul_quantize(h.cuda(), block=block)
    a = L.silu_mul(P.f64(h))
    scale = L.scale_of(L.block_amax(a, block))
    for i, top in enumerate(tops):
        rel = (abs(top) + 1 + 4) * 2.0 ** -22
        P.assert_close(out.a_scale[i], scale[i], rel * scale[i], f"scale at {top}")
        P.assert_codes(out.AQ[i:i + 1], (a / L.spread(scale, 256))[i:i + 1], rel, f"codes at {top}")
