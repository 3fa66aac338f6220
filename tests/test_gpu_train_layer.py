"""A training step of the example's layer: its gradients against fp32 torch, over micro-batches, clipped, with
block-scaled and with bf16 products, eager and captured."""
import importlib.util
import os
import sys

import pytest
import torch

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def ex():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    spec = importlib.util.spec_from_file_location("moe_layer_training", os.path.join(ROOT, "examples", "moe_layer.py"))
    m = importlib.util.module_from_spec(spec)
    sys.modules["moe_layer_training"] = m
    spec.loader.exec_module(m)
    return m


def batch(T, H, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return [torch.randn(T, H, generator=g, device="cuda").to(torch.bfloat16) for _ in range(4)]


@pytest.mark.parametrize("fp8", [True, False])
@pytest.mark.parametrize("T,H,I,E,k", [(1, 128, 128, 4, 2), (37, 256, 128, 8, 2), (300, 512, 384, 16, 4)])
def test_gradients_match_fp32(ex, T, H, I, E, k, fp8):
    """Codes are within 2^-4 of their values, about 0.026 in the root mean square; a product of two such
    operands is off by 0.037 of its own size, and each gradient here passes two or three products or codes
    after each other: about 0.065, which 0.1 bounds (bf16 products add nothing that counts)."""
    w = ex.random_weights(H, I, E, seed=T)
    q = ex.train_operands(w, fp8)
    grads = {n: torch.zeros_like(getattr(w, n)) for n in ("norm", "router", "w1", "w2")}
    want = dict.fromkeys(grads, 0.0)
    for b in (batch(T, H, T + 1), batch(T, H, T + 2)):
        x, res, dout, dres = b
        out, stream, kept = ex.train_forward(x, res, w, q, k)
        dx = ex.train_backward(dout, dres, w, q, kept, grads)
        out32, g32 = ex.reference(x, res, w, kept[2].ids.long(), dout, dres)
        assert torch.equal(stream, (x.float() + res.float()).to(torch.bfloat16))
        for name, got, ref in (("output", out, out32), ("input", dx, g32[0])):
            off = float((got.float() - ref).norm() / ref.norm())
            print(f"{name}: {off:.4f}", flush=True)
            assert off < 0.1, (name, off)
        for n, g in zip(want, g32[1:]):
            want[n] = want[n] + g
    for n in grads:
        off = float((grads[n] - want[n]).norm() / want[n].norm())
        print(f"{n}: {off:.4f}", flush=True)
        assert off < 0.1, (n, off)


@pytest.mark.parametrize("T,H,I,E,k", [(37, 256, 128, 8, 2), (300, 512, 384, 16, 4)])
def test_a_bf16_layer_holds_nothing_in_8_bits(ex, T, H, I, E, k):
    """Each gradient of the experts passes fewer than 16 roundings to bf16 after one another, each off by 2^-8 of its value at
    most and without regard to the others: 4 * 2^-8 of the whole in the root mean square.  One e4m3 operand is off by 2^-4 at
    most, 0.026 in the root mean square, and is seen."""
    w = ex.random_weights(H, I, E, seed=T)
    q = ex.train_operands(w, False)
    grads = {n: torch.zeros_like(getattr(w, n)) for n in ("norm", "router", "w1", "w2")}
    x, res, dout, dres = batch(T, H, T + 5)
    out, _, kept = ex.train_forward(x, res, w, q, k)
    dx = ex.train_backward(dout, dres, w, q, kept, grads)
    out32, g32 = ex.reference(x, res, w, kept[2].ids.long(), dout, dres)
    for name, got, ref in (("output", out, out32), ("input", dx, g32[0]), ("w1", grads["w1"], g32[3]), ("w2", grads["w2"], g32[4])):
        off = float((got.float() - ref).norm() / ref.norm())
        print(f"{name}: {off:.4f}", flush=True)
        assert off < 4 * 2.0 ** -8, (name, off)


@pytest.mark.parametrize("fp8", [True, False])
def test_step_clips_and_updates(ex, fp8):
    T, H, I, E, k = 64, 256, 128, 8, 2
    batches = [batch(T, H, s) for s in (1, 2)]
    free, clipped = (ex.random_weights(H, I, E, seed=3) for _ in range(2))
    start = {n: getattr(free, n).clone() for n in ("norm", "router", "w1", "w2")}
    g0, norm = ex.train_step(batches, free, k, lr=0.5, max_norm=float("inf"), fp8=fp8)
    want = torch.sqrt(sum((g.double() ** 2).sum() for g in g0.values()))
    # the norm: one rounding to fp32 of a sum held in 64 bits
    assert abs(norm.double() - want) <= 2.0 ** -23 * want
    bound = float(want) / 4
    g1, norm1 = ex.train_step(batches, clipped, k, lr=0.5, max_norm=bound, fp8=fp8)
    assert torch.equal(norm, norm1)
    for n in g0:
        # the factor's rounding and the product's, half a step each; the factor's eps is 1e-6 beside the norm
        scaled = g0[n].double() * (bound / (norm.double() + 1e-6))
        assert bool(((g1[n].double() - scaled).abs() <= 2.0 ** -22 * scaled.abs()).all()), n
        for weights, g in ((free, g0[n]), (clipped, g1[n])):
            assert torch.equal(getattr(weights, n), start[n].sub(g, alpha=0.5))


def test_captured_step(ex):
    """Forward and backward of one micro-batch in a graph, gradients added up over its replays."""
    T, H, I, E, k = 128, 256, 128, 8, 2
    w = ex.random_weights(H, I, E, seed=5)
    x, res, dout, dres = batch(T, H, 6)
    experts = {n: torch.zeros_like(getattr(w, n)) for n in ("w1", "w2")}
    import fp8_rowwise_scaled_amd as F
    route = F.f8f8bf16_route(torch.randn(T, E, device="cuda"), k)
    dy, _ = F.f8f8bf16_moe_combine_backward(dout, route.dst_row)

    def calls():
        q = ex.train_operands(w, True)
        rows = F.f8f8bf16_moe_combine_backward(x, route.dst_row)[0]
        h = ex.train_product(F.f8f8bf16_quantize_groupwise(rows), rows, q["w1"], route.M_sizes)
        act = F.f8f8bf16_silu_mul_quantize(h, block=128, checkpoint=True)
        da = ex.train_dgrad(dy, q["w2"], route.M_sizes)
        dh = F.f8f8bf16_silu_mul_backward(da, act.HQ, act.h_scale)
        F.bf16_grouped_stacked_wgrad(dh, rows, route.M_sizes, dW=experts["w1"], accumulate=True)
        drows = ex.train_dgrad(dh, q["w1"], route.M_sizes)
        norm = F.f8f8bf16_grad_clip([experts["w1"]], 1e9)
        return h, drows, norm

    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        calls()
    torch.cuda.current_stream().wait_stream(stream)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        captured = calls()
    for rep in range(4):
        x.copy_(torch.randn(T, H, device="cuda"))
        w.w1.mul_(1.1)
        for g in experts.values():
            g.zero_()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in (*captured, experts["w1"])]
        experts["w1"].zero_()
        want = [*calls(), experts["w1"]]
        for i, (a, b) in enumerate(zip(got, want)):
            assert torch.equal(a, b), f"replay {rep}: output {i} differs from the eager call"
