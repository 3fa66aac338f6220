"""GPU parity of the 8-bit activation checkpoints and their backward use (64-bit oracle).

Error counts (u = 2^-24): the sigmoid's exponent is off by |g| u twice over, exp2, the
sum and the reciprocal by 2 u each, the two products by u: for |g| <= 40 an activation is
known to 2^-17, its code to twice that.  A checkpoint's value is exact, its quotient and
product are one rounding each.
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


def hidden(rng, rows, I):
    h = rng.normal(0, 1, (rows, 2 * I)) * 2.0 ** rng.uniform(-3, 2, (rows, 1))
    if rows > 3:
        h[1] = 0.0
        h[2, :I] = 0.0
        h[3, 0], h[3, I - 1], h[3, I] = 40.0, -40.0, 900.0
    return P.to_bf16(np.clip(h, -900, 900) * np.where(np.arange(2 * I) < I, np.minimum(1, 40 / np.maximum(np.abs(h), 40)), 1))


CASES = [(1, 8), (5, 120), (4, 128), (6, 136), (9, 512), (7, 520), (130, 1000), (33, 2048), (5, 2056), (6, 4096), (4, 5000), (3, 8192),
         (2, 8200), (2, 14336), (1, 32768), (300, 256), (3, 1024), (2, 1032), (2, 16392)]


@pytest.mark.parametrize("rows,I", CASES)
@pytest.mark.parametrize("block", [0, 128])
def test_forward(F, rows, I, block):
    if block and I % 128:
        I = max(128, I // 128 * 128)
    print(f"case silu rows={rows} I={I} block={block}", flush=True)
    rng = np.random.default_rng(rows + I)
    h = hidden(rng, rows, I)
    nb = -(-I // 128)
    q, s = P.Guarded((rows, I), torch.uint8), P.Guarded((rows, nb) if block else (rows,), torch.float32)
    hq, hs = P.Guarded((rows, 2 * I), torch.uint8), P.Guarded((rows, 2, nb), torch.float32)
    out = F.f8f8bf16_silu_mul_quantize(h.cuda(), block=block, AQ=q.t, a_scale=s.t, HQ=hq.t, h_scale=hs.t)
    torch.cuda.synchronize()
    for g in (q, s, hq, hs):
        g.check()
    H = P.f64(h)
    act = L.silu_mul(H)
    scale = L.scale_of(L.block_amax(act, block))
    P.assert_close(out.a_scale, scale, 2.0 ** -17 * scale, "a_scale")
    P.assert_codes(out.AQ, act / L.spread(scale, I), 2.0 ** -16, "AQ")
    halves = np.split(H, 2, axis=1)
    want = np.stack([L.scale_of(L.block_amax(x, 128)) for x in halves], axis=1)
    P.assert_close(out.h_scale, want, 2.0 ** -22 * want, "h_scale")
    P.assert_codes(out.HQ, np.concatenate([x / L.spread(want[:, i], I) for i, x in enumerate(halves)], axis=1), 2.0 ** -22, "HQ")
    bare = F.f8f8bf16_silu_mul_quantize(h.cuda(), block=block)
    assert bare.HQ is None and torch.equal(bare.AQ, out.AQ) and torch.equal(bare.a_scale, out.a_scale)


@pytest.mark.parametrize("rows,I", CASES)
def test_backward(F, rows, I):
    print(f"case silu backward rows={rows} I={I}", flush=True)
    rng = np.random.default_rng(rows * 3 + I)
    ck = F.f8f8bf16_silu_mul_quantize(hidden(rng, rows, I).cuda(), checkpoint=True)
    da = P.to_bf16(rng.normal(0, 1, (rows, I)))
    out = P.Guarded((rows, 2 * I), torch.bfloat16)
    F.f8f8bf16_silu_mul_backward(da.cuda(), ck.HQ, ck.h_scale, dH=out.t)
    torch.cuda.synchronize()
    out.check()
    hs = P.f64(ck.h_scale)
    h = P.decode(ck.HQ) * np.concatenate([L.spread(hs[:, 0], I), L.spread(hs[:, 1], I)], axis=1)
    want, size = L.silu_mul_backward(P.f64(da), h)
    P.assert_close(out.t, want, P.BF16 * np.abs(want) + 2.0 ** -16 * size + 1e-38, "dH")


def test_checkpoint_gradient_is_near_the_exact_one(F):
    """Through the 8-bit checkpoint the gradient is that of the stored values: against the
    bf16 input it is off by what the codes lost (2^-4 of gate or up), no more."""
    rng = np.random.default_rng(8)
    h, da = P.to_bf16(rng.normal(0, 1, (64, 512))), P.to_bf16(rng.normal(0, 1, (64, 256)))
    ck = F.f8f8bf16_silu_mul_quantize(h.cuda(), checkpoint=True)
    got = P.f64(F.f8f8bf16_silu_mul_backward(da.cuda(), ck.HQ, ck.h_scale))
    want, _ = L.silu_mul_backward(P.f64(da), P.f64(h))
    assert np.linalg.norm(got - want) < 2.0 ** -4 * np.linalg.norm(want)


def test_no_rows(F):
    out = F.f8f8bf16_silu_mul_quantize(torch.empty((0, 32), dtype=torch.bfloat16, device="cuda"), checkpoint=True)
    assert out.AQ.shape == (0, 16) and out.HQ.shape == (0, 32)
    assert F.f8f8bf16_silu_mul_backward(torch.empty((0, 16), dtype=torch.bfloat16, device="cuda"), out.HQ, out.h_scale).shape == (0, 32)


SPLITS = [([1], 1), ([16], 16), ([128], 128), ([129], 129), ([5, 0, 300, 17], 322), ([0, 0, 7], 7), ([40, 60], 150), ([-3, 50, 90], 100),
          ([2 ** 40, 5], 33), ([130] * 70, 9100), ([0] * 5, 64), ([256, 1, 1, 254, 0], 512)]


@pytest.mark.parametrize("sizes,R", SPLITS)
@pytest.mark.parametrize("K", [16, 128, 528, 1040])
@pytest.mark.parametrize("src", ["bf16", "row", "block"])
def test_k_offsets_operand(F, sizes, R, K, src):
    if src == "block":
        K = max(128, K // 128 * 128)
    print(f"case k_offsets sizes={sizes[:6]} R={R} K={K} {src}", flush=True)
    rng = np.random.default_rng(R + K + len(sizes))
    v = rng.normal(0, 1, (R, K)) * 2.0 ** rng.uniform(-8, 8, (1, K))
    v[:, K // 2] = 0.0
    end = int(L.group_ends(sizes, R)[-1])
    v[end:] = np.nan                                     # rows of no group are not read
    xs = None
    if src == "bf16":
        x = P.to_bf16(v)
        v = P.f64(x)
    else:
        s = 2.0 ** rng.uniform(-6, 6, (R, K // 128) if src == "block" else (R,))
        xs = torch.from_numpy(s.astype(np.float32))
        codes = rng.integers(0, 0x7F, (R, K), dtype=np.uint8) | (rng.integers(0, 2, (R, K), dtype=np.uint8) << 7)
        codes[:, K // 2] = 0
        codes[end:] = 0x7F
        x = torch.from_numpy(codes)
        v = P.decode(x) * L.spread(xs.double().numpy(), K)
    v = np.where(np.arange(R)[:, None] < end, v, 0.0)
    G, cap = len(sizes), F.f8f8bf16_k_offsets_capacity(R, len(sizes))
    xt, ts, ko = P.Guarded((K, cap), torch.uint8), P.Guarded((G, K), torch.float32), P.Guarded((G,), torch.int32)
    F.f8f8bf16_quantize_k_offsets(x.cuda(), torch.tensor(sizes, dtype=torch.int64, device="cuda"),
                                  x_scale=None if xs is None else xs.cuda(), XT=xt.t, t_scale=ts.t, k_offsets=ko.t)
    torch.cuda.synchronize()
    for g in (xt, ts, ko):
        g.check()
    q, valid, scale, offs = L.k_offsets(v, sizes, cap)
    assert np.array_equal(ko.t.cpu().numpy(), offs)
    P.assert_close(ts.t, scale, 2.0 ** -22 * scale, "t_scale")
    P.assert_codes(xt.t, q, 2.0 ** -21, "codes")
    assert np.all(xt.t.cpu().numpy()[:, ~valid] == 0), "columns between and after the groups are zero"


def test_k_offsets_without_rows(F):
    xt, ts, ko = F.f8f8bf16_quantize_k_offsets(torch.empty((0, 32), dtype=torch.bfloat16, device="cuda"),
                                               torch.zeros(3, dtype=torch.int64, device="cuda"))
    assert xt.shape == (32, 0) and torch.all(ts == 1) and torch.all(ko == 0)


def test_operand_feeds_the_weight_gradient(F):
    """Both operands of the k_offsets product, made from bf16 gradients and from the fp8
    rows that the forward pass kept, against the product of what they stand for."""
    rng = np.random.default_rng(21)
    sizes, N, K = [70, 0, 129, 33], 96, 160
    R = sum(sizes)
    dy = P.to_bf16(rng.normal(0, 1, (R, N)))
    codes, xs = F.f8f8bf16_quantize_rowwise(P.to_bf16(rng.normal(0, 1, (R, K))).cuda())
    m = torch.tensor(sizes, dtype=torch.int64, device="cuda")
    at, sa, ko = F.f8f8bf16_quantize_k_offsets(dy.cuda(), m)
    bt, sb, kb = F.f8f8bf16_quantize_k_offsets(codes, m, x_scale=xs)
    assert torch.equal(ko, kb)
    dw = F.f8f8bf16_rowwise_grouped_k_offsets(at, bt, sa, sb, ko)
    torch.cuda.synchronize()
    A, B, ends = P.decode(at), P.decode(bt), ko.cpu().numpy()
    D, X = P.f64(dy), P.decode(codes) * P.f64(xs)[:, None]
    row, col = 0, 0
    for g, n in enumerate(sizes):
        a = A[:, col:ends[g]] * P.f64(sa)[g][:, None]
        b = B[:, col:ends[g]] * P.f64(sb)[g][:, None]
        want = a @ b.T
        P.assert_close(dw[g], want, P.BF16 * np.abs(want) + 2.0 ** -16 * (np.abs(a) @ np.abs(b).T) + 1e-30, f"group {g}")
        true = D[row:row + n].T @ X[row:row + n]
        # each product of two codes is off by 2^-4 + 2^-4 + 2^-8 of itself at most
        assert np.all(np.abs(want - true) <= 0.13 * (np.abs(D[row:row + n]).T @ np.abs(X[row:row + n])) + 1e-2)
        row, col = row + n, int(ends[g])


def test_offsets_past_31_bits(F):
    rows, I = 160_000, 7168                              # H holds 2.3e9 elements
    h = torch.empty((rows, 2 * I), dtype=torch.bfloat16, device="cuda")
    h.normal_()
    a = F.f8f8bf16_silu_mul_quantize(h, checkpoint=True)
    b = F.f8f8bf16_silu_mul_quantize(h[-3:].contiguous(), checkpoint=True)
    for x, y in zip(a, b):
        assert torch.equal(x[-3:], y)
    da = h[:, :I].contiguous()
    d1 = F.f8f8bf16_silu_mul_backward(da, a.HQ, a.h_scale)
    d2 = F.f8f8bf16_silu_mul_backward(da[-3:].contiguous(), b.HQ, b.h_scale)
    assert torch.equal(d1[-3:], d2)
    del h, da, d1
    R, K = 300_000, 8192
    x = torch.zeros((R, K), dtype=torch.bfloat16, device="cuda")
    x[-1000:].normal_()
    m = torch.tensor([R - 1000, 1000], dtype=torch.int64, device="cuda")
    xt, ts, ko = F.f8f8bf16_quantize_k_offsets(x, m)
    yt, us, _ = F.f8f8bf16_quantize_k_offsets(x[-1000:].contiguous(), m[1:])
    n = int(ko[0])
    assert torch.equal(xt[:, n:n + 1000], yt[:, :1000]) and torch.equal(ts[1], us[0])
