"""The training operators as a program uses them: captured in graphs with other work between the
replays, on other streams and threads, two at once, with buffers of the caller's."""
import threading

import pytest
import torch

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


def step_of(F, G, M, N, K, seed=0):
    """Inputs of one step and a function that makes all its calls on them."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    x, dy = randn(g, M, K), randn(g, M, N, sigma=0.1)
    w = torch.randn(G, N, K, generator=g, device="cuda") * K ** -0.5
    # every row in a group: rows past the last one are not written, and would hold what was there
    sizes = torch.tensor([M // G] * (G - 1) + [M - M // G * (G - 1)], dtype=torch.int64, device="cuda")
    main = torch.zeros(G, N, K, device="cuda")

    def calls():
        wb = w.to(torch.bfloat16)
        y = F.bf16_grouped_stacked(x, wb, sizes)
        dx = F.bf16_grouped_stacked_dgrad(dy, wb, sizes)
        dw = F.bf16_grouped_stacked_wgrad(dy, x, sizes)
        main.fill_(0.5)
        F.bf16_grouped_stacked_wgrad(dy, x, sizes, dW=main, accumulate=True)
        q = F.f8f8bf16_quantize_groupwise(x)
        r = F.f8f8bf16_quantize_groupwise_weight(w, transposed=True)
        total = F.f8f8bf16_grad_square_sum([dw, dx])
        norm = F.f8f8bf16_grad_clip([dw, dx], 0.01, square_sum=total)
        outs = [torch.empty_like(dw), torch.empty_like(dx)]
        norm2 = F.f8f8bf16_grad_clip([dw, dx], 1e9, outs=outs)
        return [y, dx, dw, main.clone(), *q, *r, total, norm, *outs, norm2]
    return (x, dy, w, sizes), calls


@pytest.mark.parametrize("G,M,N,K", [(4, 60, 128, 256), (2, 1200, 512, 256), (1, 6000, 128, 128), (8, 800, 256, 384)])
def test_graph_replay(F, G, M, N, K):
    (x, dy, w, sizes), calls = step_of(F, G, M, N, K)
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        calls()
    torch.cuda.current_stream().wait_stream(stream)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        captured = calls()
    scratch = torch.zeros(1 << 20, device="cuda")
    for rep in range(4):
        x.copy_(torch.randn(M, K, device="cuda"))
        dy.copy_(torch.randn(M, N, device="cuda"))
        w.mul_(1.25)
        cut = torch.randint(0, M + 1, (G - 1,)).sort().values.tolist()
        sizes.copy_(torch.tensor([b - a for a, b in zip([0] + cut, cut + [M])]))
        scratch.add_(1.0)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for i, (a, b) in enumerate(zip(captured, calls())):
            assert torch.equal(a.view(torch.uint8), b.view(torch.uint8)), f"replay {rep}: output {i} differs from the eager call"


def test_two_graphs_side_by_side(F):
    """Two captured steps, each with workspaces of its own, launched on two streams at once."""
    steps = [step_of(F, 1, 6000, 128, 128, seed=s) for s in (1, 2)]
    want = [calls() for _, calls in steps]
    torch.cuda.synchronize()
    graphs, got = [], []
    for _, calls in steps:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            got.append(calls())
        graphs.append(graph)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(5):
        for s, graph in zip(streams, graphs):
            with torch.cuda.stream(s):
                graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert all(torch.equal(p.view(torch.uint8), q.view(torch.uint8)) for p, q in zip(a, b))


def test_calls_follow_the_current_stream(F):
    (x, dy, w, sizes), calls = step_of(F, 4, 500, 256, 256, seed=5)
    want = calls()
    src = x.clone()
    x.zero_()
    big = torch.randn(4096, 4096, device="cuda")
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        for _ in range(10):
            big = big @ big * 1e-4
        x.copy_(src)
        got = calls()
    side.synchronize()
    assert all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip(got, want))


def test_calls_from_several_threads(F):
    """Each thread on a stream of its own; results as alone, errors with their own text."""
    steps = [step_of(F, 2 + i, 300 + 100 * i, 128, 256, seed=i) for i in range(4)]
    want = [calls() for _, calls in steps]
    torch.cuda.synchronize()
    failures = []

    def worker(i):
        stream = torch.cuda.Stream()
        with torch.cuda.stream(stream):
            for _ in range(20):
                got = steps[i][1]()
                stream.synchronize()
                if not all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip(got, want[i])):
                    failures.append((i, "result"))
                try:
                    F.f8f8bf16_grad_clip([steps[i][0][0]], -1.0 - i)
                    failures.append((i, "not refused"))
                except ValueError as e:
                    if f"max_norm={-1 - i}" not in str(e):
                        failures.append((i, str(e)))

    threads = [threading.Thread(target=worker, args=(i,)) for i in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not failures, failures[:3]


def test_a_workspace_serves_one_call_after_the_other(F):
    g = torch.Generator(device="cuda").manual_seed(1)
    x, dy = randn(g, 6000, 128), randn(g, 6000, 64)
    s = torch.tensor([6000], dtype=torch.int64, device="cuda")
    ws = torch.full((1 << 24,), 0xFF, dtype=torch.uint8, device="cuda")      # NaN in every type
    want = F.bf16_grouped_stacked_wgrad(dy, x, s)
    grads = [torch.randn(100000, generator=g, device="cuda"), torch.randn(77, generator=g, device="cuda")]
    norm = F.f8f8bf16_grad_square_sum(grads)
    for _ in range(3):
        assert torch.equal(F.bf16_grouped_stacked_wgrad(dy, x, s, workspace=ws), want)
        assert torch.equal(F.f8f8bf16_grad_square_sum(grads, workspace=ws), norm)
        out = torch.empty(1, device="cuda")
        assert F.f8f8bf16_grad_clip(grads, float("inf"), norm=out, workspace=ws) is not None
        assert float(out) == float(norm.sqrt().float())


def test_refused_under_capture_as_outside(F):
    """A refusal enqueues nothing: the graph around it holds what was captured before and after."""
    x = torch.ones(128, 128, dtype=torch.bfloat16, device="cuda")
    w = torch.ones(1, 128, 128, dtype=torch.bfloat16, device="cuda")
    s = torch.tensor([128], dtype=torch.int64, device="cuda")
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        a = F.bf16_grouped_stacked(x, w, s)
        with pytest.raises(ValueError):
            F.bf16_grouped_stacked(x, w, s.int())
        b = F.bf16_grouped_stacked_dgrad(a, w, s)
    for _ in range(3):
        graph.replay()
        torch.cuda.synchronize()
        assert bool((a == 128).all()) and bool((b == 128 * 128).all())
