"""GPU parity of the norm with fp8 output and its gradient (64-bit oracle).

Error counts (u = 2^-24): the sum of squares runs over at most 32 terms per thread, 6
steps in a wave and 16 waves, so it is off by at most 54 u and rstd by 30 u; h w, its
product with 448 / amax and that quotient are one rounding each (and amax is one of the
h w): a code's value is known to 4 u < 2^-21, a scale and Y's value to 40 u < 2^-18.
"""
import numpy as np
import pytest
import torch

from oracle import layer as L
from tests import layer_parity as P

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def F():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    import fp8_rowwise_scaled_amd as F
    F.load()
    return F


def rows_of(rng, rows, K, special=True):
    x = rng.normal(0, 1, (rows, K)) * 2.0 ** rng.uniform(-6, 6, (rows, 1))
    if special and rows > 3:
        x[1] = 0.0
        x[2] *= 2.0 ** -40
        x[3, K // 2] = 3000.0
    return P.to_bf16(x)


CASES = [(1, 8), (3, 16), (5, 504), (4, 512), (7, 520), (130, 1024), (33, 2048), (9, 2056), (6, 4096), (5, 4104),
         (17, 7168), (4, 7184), (3, 8192), (2, 8200), (5, 12288), (2, 32768), (300, 256), (1, 7168), (3, 1032), (2, 16384),
         (3, 16392)]


@pytest.mark.parametrize("rows,K", CASES)
@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("block", [0, 128])
def test_forward(F, rows, K, residual, block):
    if block and K % 128:
        K = max(128, K // 128 * 128)
    print(f"case norm rows={rows} K={K} residual={residual} block={block}", flush=True)
    rng = np.random.default_rng(rows * 131 + K + residual)
    x = rows_of(rng, rows, K)
    res = P.to_bf16(rng.normal(0, 1, (rows, K)) * (np.arange(rows) != 1)[:, None]) if residual else None
    wt = torch.float32 if (rows + K) % 3 else torch.bfloat16
    w = torch.from_numpy(rng.normal(1, 0.3, K).astype(np.float32)).to(wt)
    w[K // 3] = 0.0
    cols = (K // 128,) if block else ()
    q, s = P.Guarded((rows, K), torch.uint8), P.Guarded((rows, *cols), torch.float32)
    y, r = P.Guarded((rows, K), torch.bfloat16), P.Guarded((rows,), torch.float32)
    ro = P.Guarded((rows, K), torch.bfloat16) if residual else None
    out = F.f8f8bf16_rmsnorm_quantize(x.cuda(), w.cuda(), 1e-5, residual=None if res is None else res.cuda(), block=block,
                                      XQ=q.t, x_scale=s.t, Y=y.t, rstd=r.t, residual_out=ro.t if ro else None)
    torch.cuda.synchronize()
    for g in (q, s, y, r) + ((ro,) if ro else ()):
        g.check()
    h, ref, rstd = L.rmsnorm(P.f64(x), None if res is None else P.f64(res), P.f64(w), np.float64(np.float32(1e-5)))
    P.assert_close(out.rstd, rstd, 2.0 ** -18 * rstd, "rstd")
    if residual:
        assert np.array_equal(P.f64(out.residual), h)
    P.assert_close(out.Y, ref, (P.BF16 + 2.0 ** -18) * np.abs(ref) + 1e-40, "Y")
    scale = L.scale_of(L.block_amax(ref, block))
    P.assert_close(out.x_scale, scale, 2.0 ** -18 * scale, "x_scale")
    P.assert_codes(out.XQ, ref / L.spread(scale, K), 2.0 ** -21, "codes")


def test_largest_value_of_a_row_is_448(F):
    """The code of the largest magnitude is 448 itself, never the NaN above it."""
    rng = np.random.default_rng(5)
    x = P.to_bf16(rng.normal(0, 1, (2000, 264)) * 2.0 ** rng.uniform(-30, 30, (2000, 1)))
    w = torch.from_numpy(rng.normal(1, 0.3, 264).astype(np.float32))
    out = F.f8f8bf16_rmsnorm_quantize(x.cuda(), w.cuda(), 0.0)
    assert np.all(np.abs(P.decode(out.XQ)).max(axis=1) == 448.0)


def test_in_place_residual_and_optional_outputs(F):
    rng = np.random.default_rng(6)
    x, res = rows_of(rng, 5, 1040), rows_of(rng, 5, 1040)
    w = torch.ones(1040, dtype=torch.bfloat16, device="cuda")
    a = F.f8f8bf16_rmsnorm_quantize(x.cuda(), w, residual=res.cuda(), want_y=True, want_rstd=True)
    buf = res.cuda()
    b = F.f8f8bf16_rmsnorm_quantize(x.cuda(), w, residual=buf, residual_out=buf)
    assert b.Y is None and b.rstd is None and b.residual is buf
    assert torch.equal(a.XQ, b.XQ) and torch.equal(a.x_scale, b.x_scale) and torch.equal(a.residual, buf)
    c = F.f8f8bf16_rmsnorm_quantize(x.cuda(), w)
    assert c.residual is None
    e = F.f8f8bf16_rmsnorm_quantize(x.cuda()[:0], w)
    assert e.XQ.shape == (0, 1040) and e.x_scale.shape == (0,)


def test_a_bad_row_stays_alone(F):
    rng = np.random.default_rng(7)
    x = rows_of(rng, 6, 512, special=False)
    good = F.f8f8bf16_rmsnorm_quantize(x.cuda(), torch.ones(512, device="cuda"), want_y=True)
    x[2, 5], x[4, 100] = float("nan"), float("inf")
    bad = F.f8f8bf16_rmsnorm_quantize(x.cuda(), torch.ones(512, device="cuda"), want_y=True)
    keep = [0, 1, 3, 5]
    assert torch.equal(good.XQ[keep], bad.XQ[keep]) and torch.equal(good.x_scale[keep], bad.x_scale[keep])
    assert torch.equal(good.Y[keep], bad.Y[keep])


@pytest.mark.parametrize("rows,K", CASES + [(1500, 136), (700, 2048), (520, 7168)])
@pytest.mark.parametrize("residual", [False, True])
def test_backward(F, rows, K, residual):
    print(f"case norm backward rows={rows} K={K} residual={residual}", flush=True)
    rng = np.random.default_rng(rows * 17 + K + residual)
    h = rows_of(rng, rows, K)
    dy = P.to_bf16(rng.normal(0, 1, (rows, K)) * 1e-2)
    dres = P.to_bf16(rng.normal(0, 1, (rows, K)) * 1e-2) if residual else None
    wt = torch.bfloat16 if (rows + K) % 3 else torch.float32
    w = torch.from_numpy(rng.normal(1, 0.3, K).astype(np.float32)).to(wt)
    rstd = torch.from_numpy((1.0 / np.sqrt((P.f64(h) ** 2).mean(1) + 1e-5)).astype(np.float32))
    dx, dw = P.Guarded((rows, K), torch.bfloat16), P.Guarded((K,), torch.float32)
    F.f8f8bf16_rmsnorm_backward(dy.cuda(), h.cuda(), w.cuda(), rstd.cuda(), None if dres is None else dres.cuda(), dX=dx.t,
                                dweight=dw.t)
    torch.cuda.synchronize()
    dx.check()
    dw.check()
    H, DY, W, R = P.f64(h), P.f64(dy), P.f64(w), P.f64(rstd)
    want, want_w = L.rmsnorm_backward(DY, H, W, R, None if dres is None else P.f64(dres))
    xhat = H * R[:, None]
    # sums of 54 roundings, five more on the way: 2^-18 of the terms' magnitudes
    size = R[:, None] * (np.abs(DY * W) + np.abs(xhat) * np.abs(DY * W * xhat).mean(1, keepdims=True))
    size = size + (np.abs(P.f64(dres)) if residual else 0)
    P.assert_close(dx.t, want, P.BF16 * np.abs(want) + 2.0 ** -18 * size + 1e-40, "dX")
    # at most `rows` terms one after the other and 40 more steps where the parts join
    P.assert_close(dw.t, want_w, (rows + 48) * P.U * np.abs(DY * xhat).sum(0) + 1e-30, "dweight")


@pytest.mark.parametrize("K", [264, 776, 1032, 5000, 7168, 12288, 20480])
def test_backward_in_place_and_no_rows(F, K):
    rng = np.random.default_rng(9)
    h, dy, dres = (rows_of(rng, 40, K) for _ in range(3))
    w, rstd = torch.ones(K, device="cuda"), torch.rand(40, device="cuda") + 0.5
    dx, dw = F.f8f8bf16_rmsnorm_backward(dy.cuda(), h.cuda(), w, rstd, dres.cuda())
    a, b = dy.cuda(), dres.cuda()
    x1, w1 = F.f8f8bf16_rmsnorm_backward(a, h.cuda(), w, rstd, dres.cuda(), dX=a)
    x2, w2 = F.f8f8bf16_rmsnorm_backward(dy.cuda(), h.cuda(), w, rstd, b, dX=b)
    assert torch.equal(x1, dx) and torch.equal(x2, dx) and torch.equal(w1, dw) and torch.equal(w2, dw)
    _, w0 = F.f8f8bf16_rmsnorm_backward(dy.cuda()[:0], h.cuda()[:0], w, rstd[:0])
    assert torch.all(w0 == 0)


def test_offsets_past_31_bits(F):
    """Rows past element 2^31: compared with a call on those rows alone."""
    rows, K = 300_000, 7168
    x = torch.empty((rows, K), dtype=torch.bfloat16, device="cuda")
    x.normal_()
    w = torch.rand(K, device="cuda") + 0.5
    out = F.f8f8bf16_rmsnorm_quantize(x, w, block=128, want_rstd=True)
    tail = F.f8f8bf16_rmsnorm_quantize(x[-5:].contiguous(), w, block=128, want_rstd=True)
    assert torch.equal(out.XQ[-5:], tail.XQ) and torch.equal(out.x_scale[-5:], tail.x_scale)
    # a single row's gradient is the same wherever it stands
    dx, _ = F.f8f8bf16_rmsnorm_backward(x, x, w, out.rstd)
    dt, _ = F.f8f8bf16_rmsnorm_backward(x[-5:].contiguous(), x[-5:].contiguous(), w, tail.rstd)
    assert torch.equal(dx[-5:], dt)
