"""GPU parity of dispatch, combine and combine's gradients (64-bit oracle)."""
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


def places(rng, T, k, R, holes=True):
    """Distinct rows of R, some entries left out on purpose."""
    flat = np.full(T * k, -1, np.int64)
    n = min(T * k, R)
    flat[rng.permutation(T * k)[:n]] = rng.permutation(R)[:n]
    if holes:
        bad = rng.random(T * k) < 0.1
        flat[bad] = rng.choice([-1, -7, R, R + 3, 2 ** 31 - 1, -2 ** 31], bad.sum())
        flat[:k] = -1                                   # a token without any expert
    return flat.reshape(T, k)


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a, np.int32)).cuda()


@pytest.mark.parametrize("T,k,K", [(1, 1, 16), (3, 2, 32), (64, 8, 7168), (17, 4, 2064), (9, 3, 4112), (5, 64, 128), (40, 1, 9216)])
@pytest.mark.parametrize("block", [0, 128])
@pytest.mark.parametrize("holes", [False, True])
def test_dispatch(F, T, k, K, block, holes):
    if block and K % 128:
        K = max(128, K // 128 * 128)
    print(f"case dispatch T={T} k={k} K={K} block={block}", flush=True)
    rng = np.random.default_rng(T + k + K)
    R = T * k + 3
    dst = places(rng, T, k, R, holes)
    q = rng.integers(0, 256, (T, K), dtype=np.uint8)
    s = rng.random((T, K // 128) if block else (T,)).astype(np.float32)
    oq, os_ = P.Guarded((R, K), torch.uint8), P.Guarded((R, *s.shape[1:]), torch.float32)
    F.f8f8bf16_moe_dispatch(torch.from_numpy(q).cuda(), torch.from_numpy(s).cuda(), dev(dst), rows=R, XQs=oq.t, xs_out=os_.t)
    torch.cuda.synchronize()
    oq.check()
    os_.check()
    want, written = L.dispatch(q, dst, R)
    want_s, _ = L.dispatch(s, dst, R)
    assert np.array_equal(oq.t.cpu().numpy()[written], want[written])
    assert np.array_equal(os_.t.cpu().numpy()[written], want_s[written])
    assert np.all(oq.untouched(~written)) and np.all(os_.untouched(~written))


SHAPES = [(1, 1, 8), (3, 2, 16), (64, 8, 1024), (7, 9, 2056), (5, 17, 4096), (4, 64, 264), (33, 6, 7168), (6, 3, 8192), (3, 2, 8200),
          (2, 4, 20000)]


@pytest.mark.parametrize("T,k,N", SHAPES)
@pytest.mark.parametrize("weighted", [False, True])
@pytest.mark.parametrize("addend", [False, True])
def test_combine(F, T, k, N, weighted, addend):
    print(f"case combine T={T} k={k} N={N} {weighted} {addend}", flush=True)
    rng = np.random.default_rng(T * 5 + k + N)
    R = T * k + 2
    dst = places(rng, T, k, R)
    y = rng.normal(0, 1, (R, N))
    unnamed = ~np.isin(np.arange(R), dst)
    y[unnamed] = np.nan                                  # rows that no entry names are not read
    y = P.to_bf16(y)
    w = rng.normal(0, 1, (T, k)).astype(np.float32) if weighted else None
    a = P.to_bf16(rng.normal(0, 1, (T, N))) if addend else None
    out = P.Guarded((T, N), torch.bfloat16)
    F.f8f8bf16_moe_combine(y.cuda(), dev(dst), None if w is None else torch.from_numpy(w).cuda(),
                           None if a is None else a.cuda(), out=out.t)
    torch.cuda.synchronize()
    out.check()
    yy = P.f64(y)
    yy[unnamed] = 0
    want, size = L.combine(yy, dst, None if w is None else w.astype(np.float64), None if a is None else P.f64(a))
    P.assert_close(out.t, want, P.BF16 * np.abs(want) + (k + 2) * P.U * size + 1e-38, "out")
    if addend:                                          # in place
        buf = a.cuda()
        F.f8f8bf16_moe_combine(y.cuda(), dev(dst), None if w is None else torch.from_numpy(w).cuda(), buf, out=buf)
        assert torch.equal(buf, out.t)


@pytest.mark.parametrize("T,k,N", SHAPES)
@pytest.mark.parametrize("holes", [False, True])
def test_combine_backward(F, T, k, N, holes):
    print(f"case combine backward T={T} k={k} N={N}", flush=True)
    rng = np.random.default_rng(T * 3 + k + N)
    R = T * k + 2
    dst = places(rng, T, k, R, holes)
    y, dout = P.to_bf16(rng.normal(0, 1, (R, N))), P.to_bf16(rng.normal(0, 1, (T, N)))
    w = rng.normal(0, 1, (T, k)).astype(np.float32)
    dy, dw = P.Guarded((R, N), torch.bfloat16), P.Guarded((T, k), torch.float32)
    F.f8f8bf16_moe_combine_backward(dout.cuda(), dev(dst), torch.from_numpy(w).cuda(), y.cuda(), dY=dy.t, dweights=dw.t)
    torch.cuda.synchronize()
    dy.check()
    dw.check()
    want, written, want_w, size = L.combine_backward(P.f64(dout), dst, w.astype(np.float64), P.f64(y))
    P.assert_close(dy.t[torch.from_numpy(written).cuda()], want[written],
                   (P.BF16 + 2 * P.U) * np.abs(want[written]) + 1e-38, "dY")
    assert np.all(dy.untouched(~written))
    # a thread adds its columns (every 256th vector of eight) one after the other, then 6 + 4 steps
    P.assert_close(dw.t, want_w, (8 * -(-N // 2048) + 12) * P.U * size + 1e-38, "dweights")
    buf = y.cuda()                                      # dY over Y
    _, dw2 = F.f8f8bf16_moe_combine_backward(dout.cuda(), dev(dst), torch.from_numpy(w).cuda(), buf, dY=buf)
    sel = torch.from_numpy(written).cuda()
    assert torch.equal(buf[sel], dy.t[sel]) and torch.equal(dw2, dw.t)
    assert torch.equal(buf[~sel], y.cuda()[~sel])


def test_dispatch_of_bf16_rows_and_its_gradient(F):
    """Without weights: rows go out unchanged, and combine adds up what comes back."""
    rng = np.random.default_rng(3)
    x = P.to_bf16(rng.normal(0, 1, (20, 520)))
    dst = places(rng, 20, 3, 60, holes=False)
    rows, none = F.f8f8bf16_moe_combine_backward(x.cuda(), dev(dst))
    assert none is None
    want, written = L.dispatch(P.f64(x), dst, 60)
    assert np.array_equal(P.f64(rows)[written], want[written])
    back = F.f8f8bf16_moe_combine(rows, dev(dst))
    assert np.array_equal(P.f64(back), L.bf16(3 * P.f64(x)))


def test_empty_exchanges(F):
    none = torch.empty((0, 2), dtype=torch.int32, device="cuda")
    y = torch.zeros((4, 16), dtype=torch.bfloat16, device="cuda")
    assert F.f8f8bf16_moe_combine(y, none).shape == (0, 16)
    a = torch.randn(3, 16, device="cuda").to(torch.bfloat16)
    zero_k = torch.empty((3, 0), dtype=torch.int32, device="cuda")
    assert torch.equal(F.f8f8bf16_moe_combine(y, zero_k, addend=a), a)
    assert torch.all(F.f8f8bf16_moe_combine(y, zero_k) == 0)
    # no rows at all: every entry is left out
    dst = torch.zeros((3, 2), dtype=torch.int32, device="cuda")
    assert torch.equal(F.f8f8bf16_moe_combine(y[:0], dst, addend=a), a)
    _, dw = F.f8f8bf16_moe_combine_backward(a, dst, torch.ones(3, 2, device="cuda"), y[:0])
    assert torch.all(dw == 0)


def test_offsets_past_31_bits(F):
    """Rows of Y past element 2^31."""
    R, N, T, k = 300_000, 7168, 40, 4
    y = torch.empty((R, N), dtype=torch.bfloat16, device="cuda")
    y.normal_()
    g = torch.Generator(device="cuda").manual_seed(1)
    dst = (R - 1 - torch.randperm(1000, generator=g, device="cuda")[:T * k]).to(torch.int32).view(T, k)
    w = torch.rand(T, k, generator=g, device="cuda")
    rows = y[dst.long().view(-1)].contiguous()
    near = torch.arange(T * k, dtype=torch.int32, device="cuda").view(T, k)
    assert torch.equal(F.f8f8bf16_moe_combine(y, dst, w), F.f8f8bf16_moe_combine(rows, near, w))
    dout = torch.randn(T, N, generator=g, device="cuda").to(torch.bfloat16)
    dy1, dw1 = F.f8f8bf16_moe_combine_backward(dout, near, w, rows)
    dy2, dw2 = F.f8f8bf16_moe_combine_backward(dout, dst, w, y, dY=y)
    assert torch.equal(dw1, dw2) and torch.equal(dy2[dst.long().view(-1)], dy1)


def test_dispatch_past_31_bits(F):
    R, K, T, k = 300_000, 8192, 30, 3
    g = torch.Generator(device="cuda").manual_seed(3)
    q = torch.randint(0, 256, (T, K), dtype=torch.uint8, device="cuda", generator=g)
    s = torch.rand((T, K // 128), device="cuda", generator=g)
    dst = (R - 1 - torch.randperm(500, generator=g, device="cuda")[:T * k]).to(torch.int32).view(T, k)
    out, scales = F.f8f8bf16_moe_dispatch(q, s, dst, rows=R)
    assert torch.equal(out[dst.long()], q[:, None].expand(T, k, K))
    assert torch.equal(scales[dst.long()], s[:, None].expand(T, k, K // 128))
