"""GPU parity of the block-scaled products' operands with the 64-bit oracle.

u = 2^-24 is half a step of fp32.  A scale is amax (exact) times 1 / 448 rounded: 2 u.  A code's value before
its own rounding is x times 448 / amax: both round once, 2 u; 4 u covers second orders."""
import numpy as np
import pytest
import torch

from oracle import train as O
from tests import layer_parity as P

pytestmark = pytest.mark.gpu
REL = 4 * P.U


@pytest.fixture(scope="module")
def F():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    import fp8_rowwise_scaled_amd as F
    F.load()
    return F


def values(seed, *shape, dtype=torch.bfloat16):
    """Normal values over many magnitudes, a block of zeros, one of values below the scale's floor, a lone outlier."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn(*shape, generator=g, device="cuda") * torch.exp2(torch.randint(-20, 20, (*shape[:-1], 1), generator=g, device="cuda").float())
    flat = x.view(-1, 128)
    flat[0] = 0
    if len(flat) > 3:
        flat[1] *= 0
        flat[1, 7] = 2.0 ** -110
        flat[2, 100] = -3e38
    return x.to(dtype)


@pytest.mark.parametrize("rows,K", [(1, 128), (3, 256), (64, 7168), (1025, 384), (7, 128), (40000, 1280), (2, 32768)])
def test_rows(F, rows, K):
    print(f"case rows {rows} {K}", flush=True)
    x = values(rows + K, rows, K)
    q, s = P.Guarded((rows, K), torch.uint8), P.Guarded((rows, K // 128), torch.float32)
    F.f8f8bf16_quantize_groupwise(x, XQ=q.t, x_scale=s.t)
    torch.cuda.synchronize()
    q.check()
    s.check()
    want, scale = O.row_blocks(x.double())
    P.assert_close(s.t, scale.cpu().numpy(), 2 * P.U * scale.cpu().numpy(), "scale")
    P.assert_codes(q.t, want.cpu().numpy(), REL, "codes")


def bf16_blocks():
    """Blocks [n, 128] that hold every 8-bit significand under every 8-bit largest value, at 14 distances below it and at
    magnitudes from where the scale's floor acts up to the type's largest: whatever ties there are, and their neighbours."""
    blocks = []
    for top in (-112, -99, -60, 0, 40, 127):
        for below in range(1, 15):
            amax = torch.arange(128, 256, device="cuda").double() * 2.0 ** (top - 7)
            b = (torch.arange(128, 256, device="cuda").double() * 2.0 ** (top - below - 7)).repeat(128, 1)
            b[:, 1::2] *= -1
            b[torch.arange(128), torch.arange(128)] = amax
            blocks.append(b)
    return torch.cat(blocks).to(torch.bfloat16)


def fp32_blocks(seed):
    """Blocks [n, 128, 128] of fp32 values at the middles of two codes, and one step of fp32 to either side."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    table = torch.tensor(O.E4M3_MAGNITUDES, dtype=torch.float64, device="cuda")
    n = 64
    amax = (1 + torch.rand(n, 1, generator=g, device="cuda").double()).float()
    amax[::4] = (amax[::4] * 16).round() / 16                  # few bits: many exact ties
    amax[1::4] = amax[1::4].to(torch.bfloat16).float()
    amax = amax * torch.exp2(torch.randint(-99, 127, (n, 1), generator=g, device="cuda").float())
    i = torch.randint(0, 126, (n, 128 * 128), generator=g, device="cuda")
    v = ((table[i] + table[i + 1]) / 2 * amax.double() / 448).float()
    v = (v.contiguous().view(torch.int32) + torch.randint(-1, 2, v.shape, generator=g, device="cuda", dtype=torch.int32)).view(torch.float32)
    v = torch.where(v.abs() <= amax, v, 0.0) * (1 - 2 * (i % 2))
    v[:, 77] = amax[:, 0]
    return v.view(n, 128, 128)


def test_every_code_is_the_nearest(F):
    """No tolerance: the quotient by the real amax / 448, ties to the even code, decided in exact arithmetic."""
    x = bf16_blocks()
    amax = x.double().abs().amax(1, keepdim=True)
    q, _ = F.f8f8bf16_quantize_groupwise(x)
    wrong = ~O.nearest(q, x.double(), amax)
    assert not bool(wrong.any()), f"rows: {int(wrong.sum())} codes, first at {wrong.nonzero()[0].tolist()}"
    w = x.view(-1, 128, 128).clone()
    for at, t in (("bf16", w), ("fp32 of bf16", w.float())):
        amax = t.double().abs().amax((1, 2), keepdim=True)
        q = F.f8f8bf16_quantize_groupwise_weight(t).WQ
        wrong = ~O.nearest(q, t.double(), amax)
        assert not bool(wrong.any()), f"weights, {at}: {int(wrong.sum())} codes, first at {wrong.nonzero()[0].tolist()}"
    for seed in range(8):
        w = fp32_blocks(seed)
        r = F.f8f8bf16_quantize_groupwise_weight(w, transposed=True)
        wrong = ~O.nearest(r.WQ, w.double(), w.double().abs().amax((1, 2), keepdim=True))
        assert not bool(wrong.any()), f"fp32 weights, seed {seed}: {int(wrong.sum())} codes, first at {wrong.nonzero()[0].tolist()}"


def test_rows_agree_with_the_rowwise_quantiser(F):
    """One block per row: the codes of f8f8bf16_quantize_rowwise, but for values within rounding of a midpoint."""
    x = torch.randn(500, 128, device="cuda").to(torch.bfloat16)
    a, sa = F.f8f8bf16_quantize_groupwise(x)
    b, sb = F.f8f8bf16_quantize_rowwise(x)
    assert bool(((sa[:, 0] - sb).abs() <= 2 * P.U * sb * 1.01).all())
    # Both place a value by an fp32 quotient that is off by at most 4 u; where they differ, the exact one lies that
    # near to the middle of their codes.  (How many there are says nothing: 8-bit values over 8-bit scales often
    # hit a middle exactly.)
    va, vb = a.view(torch.float8_e4m3fn).double(), b.view(torch.float8_e4m3fn).double()
    exact = x.double() / (x.double().abs().amax(1, keepdim=True) / 448)
    off = va != vb
    assert bool(((exact - (va + vb) / 2).abs()[off] <= REL * exact.abs()[off]).all())


@pytest.mark.parametrize("G,N,K", [(1, 128, 128), (2, 256, 128), (3, 128, 384), (2, 512, 1024), (5, 256, 256)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("turned", [False, True])
def test_weights(F, G, N, K, dtype, turned):
    print(f"case weights {G} {N} {K} {dtype} {turned}", flush=True)
    w = values(G + N + K, G, N, K, dtype=dtype)
    out = [P.Guarded((G, N, K), torch.uint8), P.Guarded((G, N // 128, K // 128), torch.float32)]
    if turned:
        out += [P.Guarded((G, K, N), torch.uint8), P.Guarded((G, K // 128, N // 128), torch.float32)]
    r = F.f8f8bf16_quantize_groupwise_weight(w, turned, *(o.t for o in out))
    torch.cuda.synchronize()
    for o in out:
        o.check()
    want, scale = O.weight_blocks(w.double())
    P.assert_close(r.w_scale, scale.cpu().numpy(), 2 * P.U * scale.cpu().numpy(), "scale")
    P.assert_codes(r.WQ, want.cpu().numpy(), REL, "codes")
    if turned:
        assert torch.equal(r.WQt, r.WQ.transpose(1, 2)) and torch.equal(r.wt_scale, r.w_scale.transpose(1, 2))
    else:
        assert r.WQt is None and r.wt_scale is None


def test_every_byte_of_a_block_is_turned(F):
    """All 128 x 128 places of a block told apart: 254 finite codes, each at many places."""
    codes = torch.tensor([c for c in range(256) if c & 0x7F != 0x7F], dtype=torch.uint8).view(torch.float8_e4m3fn).float()
    w = codes[torch.randint(0, 254, (1, 128, 128), generator=torch.Generator().manual_seed(1))].cuda()
    w[0, 0, 0] = 448.0
    r = F.f8f8bf16_quantize_groupwise_weight(w, transposed=True)
    assert torch.equal(r.WQ.view(torch.float8_e4m3fn).float(), w) and torch.equal(r.WQt, r.WQ.transpose(1, 2))
    assert bool((r.w_scale - 1).abs() <= 2 * P.U)


def test_a_nan_stays_in_its_block(F):
    x = values(3, 8, 512)
    clean = F.f8f8bf16_quantize_groupwise(x)
    w = values(4, 1, 256, 256, dtype=torch.float32)
    wc = F.f8f8bf16_quantize_groupwise_weight(w, transposed=True)
    for bad in (float("nan"), float("inf")):
        y = x.clone()
        y[3, 200] = bad
        q, s = F.f8f8bf16_quantize_groupwise(y)
        keep = torch.ones(8, 4, dtype=torch.bool, device="cuda")
        keep[3, 1] = False
        assert torch.equal(s[keep], clean[1][keep]) and torch.equal(q.view(8, 4, 128)[keep], clean[0].view(8, 4, 128)[keep])
        v = w.clone()
        v[0, 10, 140] = bad
        r = F.f8f8bf16_quantize_groupwise_weight(v, transposed=True)
        for a, b in ((r.WQ, wc.WQ), (r.WQt.transpose(1, 2), wc.WQt.transpose(1, 2))):
            assert torch.equal(a[0, :, :128], b[0, :, :128]) and torch.equal(a[0, 128:], b[0, 128:])


def test_offsets_past_31_bits(F):
    rows, K = 66000, 32768
    x = torch.zeros(rows, K, dtype=torch.bfloat16, device="cuda")
    x[-3:] = values(1, 3, K)
    q, s = F.f8f8bf16_quantize_groupwise(x)
    want = F.f8f8bf16_quantize_groupwise(x[-3:].contiguous())
    assert torch.equal(q[-3:], want[0]) and torch.equal(s[-3:], want[1]) and bool((s[:-3] == 1).all()) and not (q[:-3] & 0x7F).any()
    del x, q, s
    w = torch.zeros(3, 32768, 32768, dtype=torch.bfloat16, device="cuda")
    w[2, -128:, -256:] = values(2, 128, 256)
    r = F.f8f8bf16_quantize_groupwise_weight(w, transposed=True)
    want = F.f8f8bf16_quantize_groupwise_weight(w[2, -128:, -256:].contiguous(), transposed=True)
    assert torch.equal(r.WQ[2, -128:, -256:], want.WQ) and torch.equal(r.WQt[2, -256:, -128:], want.WQt)
    assert torch.equal(r.w_scale[2, -1, -2:], want.w_scale[0]) and torch.equal(r.wt_scale[2, -2:, -1], want.wt_scale[:, 0])


@pytest.mark.parametrize("G,M,N,K", [(2, 100, 256, 384), (4, 700, 512, 256)])
def test_operands_of_the_block_scaled_product(F, G, M, N, K):
    """Both directions of a product on these operands: the library's product of the codes against fp64
    from the same codes (its own tolerance), so the operands' layouts are what it reads."""
    g = torch.Generator(device="cuda").manual_seed(M)
    x = torch.randn(M, K, generator=g, device="cuda").to(torch.bfloat16)
    dy = torch.randn(M, N, generator=g, device="cuda").to(torch.bfloat16)
    w = torch.randn(G, N, K, generator=g, device="cuda")
    sizes = torch.tensor([M - 10 * (G - 1)] + [10] * (G - 1), dtype=torch.int64, device="cuda")
    r = F.f8f8bf16_quantize_groupwise_weight(w, transposed=True)
    for rows, wq, ws in ((x, r.WQ, r.w_scale), (dy, r.WQt, r.wt_scale)):
        q, s = F.f8f8bf16_quantize_groupwise(rows)
        got = F.f8f8bf16_groupwise_grouped_stacked(q, wq, s, ws, sizes).double()
        qv = q.view(torch.float8_e4m3fn).double() * s.double().repeat_interleave(128, 1)
        wv = wq.view(torch.float8_e4m3fn).double() * ws.double().repeat_interleave(128, 1).repeat_interleave(128, 2)
        want, size, _ = O.forward(qv, wv, sizes.tolist())
        assert bool(((got - want).abs() <= 2.0 ** -8 * want.abs() + (q.shape[1] + 8) * 2.0 ** -24 * size).all())


def test_binding(F):
    x = torch.randn(8, 256, device="cuda").to(torch.bfloat16)
    w = torch.randn(128, 256, device="cuda")
    r = F.f8f8bf16_quantize_groupwise_weight(w, transposed=True)
    assert r.WQ.shape == (128, 256) and r.w_scale.shape == (1, 2) and r.WQt.shape == (256, 128) and r.wt_scale.shape == (2, 1)
    buf = torch.empty((8, 256), dtype=torch.float8_e4m3fn, device="cuda")
    q, _ = F.f8f8bf16_quantize_groupwise(x, XQ=buf)
    assert q.dtype is torch.uint8 and q.data_ptr() == buf.data_ptr()
    empty = F.f8f8bf16_quantize_groupwise(x[:0])
    assert empty[0].shape == (0, 256) and empty[1].shape == (0, 2)
    none = F.f8f8bf16_quantize_groupwise_weight(w[None][:0], transposed=True)
    assert none.WQ.shape == (0, 128, 256) and none.WQt.shape == (0, 256, 128)
    for call, text in [
            (lambda: F.f8f8bf16_quantize_groupwise(x[:, :200].contiguous()), "128"),
            (lambda: F.f8f8bf16_quantize_groupwise(x.t()), "contiguous|128"),
            (lambda: F.f8f8bf16_quantize_groupwise(x, x_scale=torch.empty(8, device="cuda")), "shape"),
            (lambda: F.f8f8bf16_quantize_groupwise_weight(w[:100].contiguous()), "128"),
            (lambda: F.f8f8bf16_quantize_groupwise_weight(w[0]), r"\[G, N, K\]"),
            (lambda: F.f8f8bf16_quantize_groupwise_weight(w, WQ=torch.empty((256, 128), dtype=torch.uint8, device="cuda")), "shape"),
            (lambda: F.f8f8bf16_quantize_groupwise_weight(w, WQ=w.view(torch.uint8)[:, :256]), "contiguous|overlaps")]:
        with pytest.raises(ValueError, match=text):
            call()
    assert np.isfinite(P.decode(q)).all()
