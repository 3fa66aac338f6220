"""The operators together: the example's layer against fp32 torch, under graph replay, on
another stream, and from several threads."""
import importlib.util
import os
import threading

import pytest
import torch

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def ex():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    spec = importlib.util.spec_from_file_location("moe_layer_example", os.path.join(ROOT, "examples", "moe_layer.py"))
    m = importlib.util.module_from_spec(spec)
    import sys
    sys.modules["moe_layer_example"] = m
    spec.loader.exec_module(m)
    return m


def inputs(T, H, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return [torch.randn(T, H, generator=g, device="cuda").to(torch.bfloat16) for _ in range(4)]


@pytest.mark.parametrize("T,H,I,E,k", [(1, 128, 64, 4, 2), (37, 256, 128, 8, 2), (300, 512, 320, 16, 4)])
def test_layer_matches_fp32(ex, T, H, I, E, k):
    """A code is within 2^-4 of its value, about 0.026 in the root mean square; a product of
    two such operands is off by 0.037 of its own size, and each output here passes two
    or three products or codes after each other: about 0.065.  0.1 bounds that, and a
    wrong term or a misplaced row is far outside."""
    w = ex.random_weights(H, I, E, seed=T)
    q = w.quantized()
    x, res, dout, dres = inputs(T, H, T + 1)
    out, stream, kept = ex.forward(x, res, w, q, k)
    grads = ex.backward(dout, dres, w, q, kept)
    want, want_grads = ex.reference(x, res, w, kept[2].ids.long(), dout, dres)
    assert torch.equal(stream, (x.float() + res.float()).to(torch.bfloat16))
    for name, got, ref in zip(("output", "input", "norm", "router", "w1", "w2"), (out, *grads), (want, *want_grads)):
        off = float((got.float() - ref).norm() / ref.norm())
        print(f"{name}: {off:.4f}", flush=True)
        assert off < 0.1, (name, off)


def flat(result):
    """All tensors of nested tuples, in order."""
    if isinstance(result, torch.Tensor):
        return [result]
    return [t for r in result if r is not None for t in flat(r)]


def test_layer_under_graph_replay(ex):
    """Both passes' library calls captured in one graph and replayed with eager work and
    synchronisations in between, on inputs that change between the replays."""
    import fp8_rowwise_scaled_amd as F
    T, H, I, E, k = 200, 256, 128, 8, 2
    w = ex.random_weights(H, I, E, seed=3)
    q = w.quantized()
    x, res, dout, dres = inputs(T, H, 4)
    logits = torch.randn(T, E, device="cuda")

    def calls():
        norm = F.f8f8bf16_rmsnorm_quantize(x, w.norm, residual=res, want_y=True, want_rstd=True)
        route = F.f8f8bf16_route(logits, k, bias=w.bias, score="sigmoid", n_group=4, topk_group=2, group_top=2)
        rows, scales = F.f8f8bf16_moe_dispatch(norm.XQ, norm.x_scale, route.dst_row)
        h = F.f8f8bf16_rowwise_grouped_stacked(rows, q["w1"][0], scales, q["w1"][1], route.M_sizes)
        act = F.f8f8bf16_silu_mul_quantize(h, checkpoint=True)
        y = F.f8f8bf16_rowwise_grouped_stacked(act.AQ, q["w2"][0], act.a_scale, q["w2"][1], route.M_sizes)
        out = F.f8f8bf16_moe_combine(y, route.dst_row, route.weights)
        dy, dw = F.f8f8bf16_moe_combine_backward(dout, route.dst_row, route.weights, y)
        xt = F.f8f8bf16_quantize_k_offsets(rows, route.M_sizes, x_scale=scales)
        dh = F.f8f8bf16_silu_mul_backward(dy[:, :I].contiguous(), act.HQ, act.h_scale)
        dl = F.f8f8bf16_route_backward(logits, route.ids, dw, score="sigmoid")
        back = F.f8f8bf16_rmsnorm_backward(dout, norm.residual, w.norm, norm.rstd, dresidual=dres)
        return flat((norm, route, rows, scales, h, act, y, out, dy, dw, xt, dh, dl, back))

    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        calls()
    torch.cuda.current_stream().wait_stream(stream)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=stream):
        captured = calls()
    scratch = torch.zeros(1 << 20, device="cuda")
    for rep in range(4):
        logits.copy_(torch.randn(T, E, device="cuda"))
        x.copy_(torch.randn(T, H, device="cuda"))
        scratch.add_(1.0)
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        for i, (a, b) in enumerate(zip(captured, calls())):
            assert torch.equal(a.view(torch.uint8), b.view(torch.uint8)), f"replay {rep}: output {i} differs from the eager call"


def test_calls_follow_the_current_stream(ex):
    """Work queued on a side stream behind a long computation of its input."""
    import fp8_rowwise_scaled_amd as F
    x = torch.zeros((64, 1024), dtype=torch.bfloat16, device="cuda")
    w = torch.ones(1024, device="cuda")
    src = torch.randn(64, 1024, device="cuda").to(torch.bfloat16)
    want = F.f8f8bf16_rmsnorm_quantize(src, w)
    big = torch.randn(4096, 4096, device="cuda")
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        for _ in range(10):
            big = big @ big * 1e-4
        x.copy_(src)
        got = F.f8f8bf16_rmsnorm_quantize(x, w)
    side.synchronize()
    assert torch.equal(got.XQ, want.XQ) and torch.equal(got.x_scale, want.x_scale)


def test_calls_from_several_threads(ex):
    """Each thread on a stream of its own; results as alone, errors with their own text."""
    import fp8_rowwise_scaled_amd as F
    xs = [torch.randn(300, 64, device="cuda") for _ in range(4)]
    want = [F.f8f8bf16_route(x, 4) for x in xs]
    torch.cuda.synchronize()
    failures = []

    def worker(i):
        stream = torch.cuda.Stream()
        with torch.cuda.stream(stream):
            for _ in range(50):
                r = F.f8f8bf16_route(xs[i], 4)
                stream.synchronize()
                if not all(torch.equal(a, b) for a, b in zip(r, want[i])):
                    failures.append((i, "result"))
                try:
                    F.f8f8bf16_route(xs[i], 17 + i)
                    failures.append((i, "not refused"))
                except ValueError as e:
                    if f"k={17 + i}" not in str(e):
                        failures.append((i, str(e)))

    threads = [threading.Thread(target=worker, args=(i,)) for i in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not failures, failures[:3]


def test_buffers_and_refusals_of_the_binding(ex):
    import fp8_rowwise_scaled_amd as F
    x = torch.randn(8, 256, device="cuda").to(torch.bfloat16)
    w = torch.ones(256, device="cuda")
    # float8 buffers are taken where codes are, and come back as their bytes
    buf = torch.empty((8, 256), dtype=torch.float8_e4m3fn, device="cuda")
    r = F.f8f8bf16_rmsnorm_quantize(x, w, XQ=buf)
    assert r.XQ.data_ptr() == buf.data_ptr() and r.XQ.dtype == torch.uint8
    ids = torch.zeros((8, 1), dtype=torch.int32, device="cuda")
    ids[:, 0] = torch.arange(8)
    q, _ = F.f8f8bf16_moe_dispatch(buf, r.x_scale, ids)
    assert torch.equal(q, r.XQ)
    for call, text in [
            (lambda: F.f8f8bf16_rmsnorm_quantize(x.t(), w), "contiguous"),
            (lambda: F.f8f8bf16_rmsnorm_quantize(x, w[:-8]), "shape"),
            (lambda: F.f8f8bf16_rmsnorm_quantize(x, w, residual_out=x), "without a residual"),
            (lambda: F.f8f8bf16_rmsnorm_quantize(x, w, block=64), "block"),
            (lambda: F.f8f8bf16_rmsnorm_quantize(x, w, Y=x), "overlaps"),
            (lambda: F.f8f8bf16_rmsnorm_quantize(x, w, XQ=torch.empty((8, 256), device="cuda")), "uint8"),
            (lambda: F.f8f8bf16_rmsnorm_quantize(x, w, rstd=torch.empty(8)), "on the GPU"),
            (lambda: F.f8f8bf16_route(x, 2, score="relu"), "softmax"),
            (lambda: F.f8f8bf16_route(x, 2, plan=False, M_sizes=torch.empty(256, dtype=torch.int64, device="cuda")), "plan"),
            (lambda: F.f8f8bf16_route(x, 2, n_group=3), "n_group"),
            (lambda: F.f8f8bf16_route(x, -1), "negative"),
            (lambda: F.f8f8bf16_moe_combine(x, ids.long()), "int32"),
            (lambda: F.f8f8bf16_moe_combine_backward(x, ids, None, x, rows=9), "rows=9"),
            (lambda: F.f8f8bf16_silu_mul_quantize(x[:, :255].contiguous()), "even number"),
            (lambda: F.f8f8bf16_quantize_k_offsets(x, torch.ones(2, device="cuda")), "int64"),
            (lambda: F.f8f8bf16_quantize_k_offsets(x, torch.ones(2, dtype=torch.int64, device="cuda"),
                                                   workspace=torch.empty(8, device="cuda")), "workspace"),
            (lambda: F.f8f8bf16_rmsnorm_quantize(None, w), "tensor")]:
        with pytest.raises(ValueError, match=text):
            call()
    class Undecided:
        def __bool__(self):
            raise KeyError("undecided")
    with pytest.raises(KeyError, match="undecided"):
        F.f8f8bf16_rmsnorm_quantize(x, w, want_y=Undecided())
    with pytest.raises(TypeError):
        F.f8f8bf16_rmsnorm_quantize(x, w, eps="small")
