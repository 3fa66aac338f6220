"""Cases that measure the operators for training the experts: products in bf16, operands of the
block-scaled products, the gradients' norm.

    products       bf16_grouped_stacked, bf16_grouped_stacked_dgrad, bf16_grouped_stacked_wgrad
    block scales   f8f8bf16_quantize_groupwise, f8f8bf16_quantize_groupwise_weight
    clipping       f8f8bf16_grad_clip, f8f8bf16_grad_square_sum

With ``own`` false ``run`` computes an operator from elementary torch operations,
with ``own`` true it makes the library's call.  Sizes: gate and up (N = 4096, K = 7168), down
(N = 7168, K = 2048) and the tails (N = 1000, K = 7184) are those of the grouped GEMM workloads of
this repository; the others are generic.
"""
import math
import random

import torch

own = False

E4M3_MAX = 448.0
FP8 = torch.float8_e4m3fn
BLOCK = 128


def listed():
    return [
        # serving: one token, one of eight experts' down product, bound by reading one weight
        {"name": "product_one_token", "kind": "fwd", "G": 8, "M": 1, "N": 7168, "K": 2048},
        # a training batch's gate and up product, skewed sizes
        {"name": "product_train", "kind": "fwd", "G": 8, "M": 4096, "N": 4096, "K": 7168},
        # the gradient of its input, from the weights as the forward pass holds them
        {"name": "dgrad_train", "kind": "dgrad", "G": 8, "M": 4096, "N": 4096, "K": 7168},
        # odd rows over many experts, some without any, N and K with tails
        {"name": "dgrad_tails", "kind": "dgrad", "G": 16, "M": 1537, "N": 1000, "K": 7184},
        # the gradient of its weights, kept in fp32
        {"name": "wgrad_train", "kind": "wgrad", "G": 8, "M": 4096, "N": 4096, "K": 7168, "out": "f32"},
        # many small experts, odd rows, gradients in bf16
        {"name": "wgrad_many", "kind": "wgrad", "G": 64, "M": 6143, "N": 1024, "K": 1536, "out": "bf16"},
        # rows of a gradient made the operand of a block-scaled product: a small batch, and a large odd one
        {"name": "rows_small", "kind": "rows", "rows": 64, "K": 7168},
        {"name": "rows_train", "kind": "rows", "rows": 16383, "K": 4096},
        # weights requantised after an optimizer's step: fp32 masters for both products that read them; a small bf16 one for inference
        {"name": "weights_train", "kind": "weight", "G": 8, "N": 4096, "K": 7168, "w": "f32", "t": True},
        {"name": "weights_small", "kind": "weight", "G": 1, "N": 2048, "K": 1024, "w": "bf16", "t": False},
        # a small model's gradients below the bound: the norm alone, in place
        {"name": "clip_small", "kind": "clip", "tensors": 12, "elements": 1_000_000, "clipped": False},
        # a layer's gradients, fp32 expert weights and bf16 others, above the bound: scaled into the buffer that the optimizer reads
        {"name": "clip_layer", "kind": "clip", "tensors": 48, "elements": 270_000_000, "clipped": True},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    """One more case: sizes over the logarithm of their range, odd rows, widths in whole 16-byte granules (whole blocks where scales need them)."""
    kind = rng.choice(["fwd", "fwd", "dgrad", "dgrad", "wgrad", "wgrad", "rows", "weight", "clip"])
    most = 200_000_000                       # elements of one tensor, below the largest listed case
    if kind in ("fwd", "dgrad", "wgrad"):
        N, K = 8 * _log(rng, 16, 1000), 8 * _log(rng, 16, 1000)
        G = min(_log(rng, 1, 128), max(1, most // (N * K)))
        M = min(_log(rng, 1, 12000), 110_000_000_000 // (N * K))
        return {"kind": kind, "G": G, "M": M, "N": N, "K": K, **({"out": rng.choice(["f32", "bf16"])} if kind == "wgrad" else {})}
    if kind == "rows":
        K = BLOCK * _log(rng, 1, 96)
        return {"kind": kind, "rows": min(_log(rng, 1, 40000), 65_000_000 // K), "K": K}
    if kind == "weight":
        N, K = BLOCK * _log(rng, 1, 64), BLOCK * _log(rng, 1, 64)
        return {"kind": kind, "G": min(_log(rng, 1, 64), max(1, most // (N * K))), "N": N, "K": K, "w": rng.choice(["bf16", "f32"]),
                "t": rng.random() < 0.6}
    return {"kind": kind, "tensors": _log(rng, 1, 200), "elements": _log(rng, 1000, most), "clipped": rng.random() < 0.6}


# ---------------------------------------------------------------- inputs

def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return g


def _normal(g, *shape, sigma=1.0):
    return torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32) * sigma


def _acts(g, rows, K):
    """Hidden states: normal, with a few channels several times larger and rows of different size."""
    x = _normal(g, rows, K)
    x *= 1.0 + 7.0 * (torch.rand(K, generator=g, device="cuda") < 0.01)
    x *= torch.exp(0.5 * _normal(g, rows, 1))
    return x.to(torch.bfloat16)


def _grads(g, rows, K):
    """Gradients of rows: small, some rows much smaller than others."""
    return (_normal(g, rows, K, sigma=1e-2) * torch.exp(_normal(g, rows, 1))).to(torch.bfloat16)


def _weights(g, G, N, K, dtype):
    w = torch.empty(G, N, K, device="cuda", dtype=dtype)
    for e in range(G):
        w[e] = _normal(g, N, K, sigma=K ** -0.5)
    return w


def _group_rows(G, M):
    """Rows per expert: skewed, an expert now and then empty."""
    r = random.Random(G * 1_000_003 + M)
    p = [r.expovariate(1.0) * (r.random() > 0.1) + 1e-9 for _ in range(G)]
    cuts, run_sum = [0], 0.0
    for v in p:
        run_sum += v
        cuts.append(round(M * run_sum / sum(p)))
    cuts[-1] = M
    return [b - a for a, b in zip(cuts, cuts[1:])]


def _tensor_sizes(n, elements):
    """Sizes of a model's gradients: most elements in a few weights, the rest down to a few values; odd ones among them."""
    r = random.Random(n * 1_000_003 + elements)
    p = [math.exp(r.gauss(0.0, 3.0)) for _ in range(n)]
    return [max(1, int(elements * v / sum(p))) for v in p]


def prepare(case, seed):
    g, c, kind = _gen(seed), dict(case), case["kind"]
    s = {"case": c}
    if kind in ("fwd", "dgrad", "wgrad"):
        s["rows"] = _group_rows(c["G"], c["M"])
        random.Random(seed).shuffle(s["rows"])
        s["sizes"] = torch.tensor(s["rows"], dtype=torch.int64, device="cuda")
        if kind != "wgrad":
            s["w"] = _weights(g, c["G"], c["N"], c["K"], torch.bfloat16)
        if kind != "dgrad":
            s["x"] = _acts(g, c["M"], c["K"])
        if kind != "fwd":
            s["dy"] = _grads(g, c["M"], c["N"])
    elif kind == "rows":
        s["x"] = _grads(g, c["rows"], c["K"])
    elif kind == "weight":
        s["w"] = _weights(g, c["G"], c["N"], c["K"], torch.float32 if c["w"] == "f32" else torch.bfloat16)
    else:
        # One flat buffer per type, as an optimizer keeps its gradients, and a tensor in it for each parameter: the larger ones fp32.
        sizes = _tensor_sizes(c["tensors"], c["elements"])
        bound = sorted(sizes)[len(sizes) // 2]
        s["flat"], s["out"], s["grads"], s["outs"] = [], [], [], []
        for dtype in (torch.float32, torch.bfloat16):
            mine = [n for n in sizes if (n >= bound) == (dtype == torch.float32)]
            flat = torch.empty(sum(mine), device="cuda", dtype=dtype)
            for part in flat.split(1 << 26):
                part.copy_(_normal(g, part.numel(), sigma=1e-3))
            out = torch.empty_like(flat) if c["clipped"] else flat
            s["flat"].append(flat)
            s["out"].append(out)
            s["grads"] += flat.split(mine)
            s["outs"] += out.split(mine)
        # the norm is close to 1e-3 sqrt(elements)
        s["max_norm"] = 1e-3 * math.sqrt(sum(sizes)) * (0.3 if c["clipped"] else 3.0)
    return s


# ---------------------------------------------------------------- one pass

def run(state):
    if own:
        import fp8_rowwise_scaled_amd as F
        return _OWN[state["case"]["kind"]](F, state, state["case"])
    return _PLAIN[state["case"]["kind"]](state, state["case"])


def _dtype(c):
    return torch.float32 if c["out"] == "f32" else torch.bfloat16


def _own_fwd(F, s, c):
    return F.bf16_grouped_stacked(s["x"], s["w"], s["sizes"])


def _own_dgrad(F, s, c):
    return F.bf16_grouped_stacked_dgrad(s["dy"], s["w"], s["sizes"])


def _own_wgrad(F, s, c):
    return F.bf16_grouped_stacked_wgrad(s["dy"], s["x"], s["sizes"], dtype=_dtype(c))


def _own_rows(F, s, c):
    q, sc = F.f8f8bf16_quantize_groupwise(s["x"])
    return {"codes": q.view(FP8), "scale": sc}


def _own_weight(F, s, c):
    r = F.f8f8bf16_quantize_groupwise_weight(s["w"], transposed=c["t"])
    return {"codes": r.WQ.view(FP8), "scale": r.w_scale, **({"codes_t": r.WQt.view(FP8), "scale_t": r.wt_scale} if c["t"] else {})}


def _own_clip(F, s, c):
    norm = F.f8f8bf16_grad_clip(s["grads"], s["max_norm"], outs=s["outs"])
    return {"norm": norm, "f32": s["out"][0], "bf16": s["out"][1]}


_OWN = {"fwd": _own_fwd, "dgrad": _own_dgrad, "wgrad": _own_wgrad, "rows": _own_rows, "weight": _own_weight, "clip": _own_clip}


def _plain_fwd(s, c):
    return torch.cat([x.float() @ w.float().t() for x, w in zip(s["x"].split(s["rows"]), s["w"]) if len(x)]).to(torch.bfloat16)


def _plain_dgrad(s, c):
    return torch.cat([d.float() @ w.float() for d, w in zip(s["dy"].split(s["rows"]), s["w"]) if len(d)]).to(torch.bfloat16)


def _plain_wgrad(s, c):
    parts = zip(s["dy"].float().split(s["rows"]), s["x"].float().split(s["rows"]))
    return torch.stack([(d.t() @ x).to(_dtype(c)) for d, x in parts])


def _plain_codes(v, dims):
    amax = v.abs().amax(dims, keepdim=True)
    sc = torch.where(amax > 0, amax / E4M3_MAX, 1.0)
    return (v / sc).clamp(-E4M3_MAX, E4M3_MAX).to(FP8), sc


def _plain_rows(s, c):
    q, sc = _plain_codes(s["x"].float().view(c["rows"], -1, BLOCK), 2)
    return {"codes": q.view(c["rows"], c["K"]), "scale": sc.squeeze(2)}


def _plain_weight(s, c):
    G, N, K = c["G"], c["N"], c["K"]
    q, sc = _plain_codes(s["w"].float().view(G, N // BLOCK, BLOCK, K // BLOCK, BLOCK), (2, 4))
    q, sc = q.view(G, N, K), sc.view(G, N // BLOCK, K // BLOCK)
    t = {"codes_t": q.view(torch.uint8).transpose(1, 2).contiguous().view(FP8), "scale_t": sc.transpose(1, 2).contiguous()} if c["t"] else {}
    return {"codes": q, "scale": sc, **t}


def _plain_clip(s, c):
    # Squares in 64 bits: the sum is a long one.
    norm = torch.stack([g.double().square().sum() for g in s["grads"]]).sum().sqrt()
    factor = (s["max_norm"] / (norm + 1e-6)).clamp(max=1.0).float()
    for flat, out in zip(s["flat"], s["out"]):
        out.copy_(flat.float() * factor)
    return {"norm": norm.float().view(1), "f32": s["out"][0], "bf16": s["out"][1]}


_PLAIN = {"fwd": _plain_fwd, "dgrad": _plain_dgrad, "wgrad": _plain_wgrad, "rows": _plain_rows, "weight": _plain_weight, "clip": _plain_clip}


# ---------------------------------------------------------------- what a pass cannot do without

def work(case):
    c, kind = case, case["kind"]
    if kind in ("fwd", "dgrad", "wgrad"):
        M, N, K = c["M"], c["N"], c["K"]
        if kind == "wgrad":
            weights = c["G"] * N * K * (4 if c["out"] == "f32" else 2)
        else:
            weights = sum(m > 0 for m in _group_rows(c["G"], M)) * N * K * 2
        return {"bytes": weights + 2 * M * (N + K) + 8 * c["G"], "flops": 2 * M * N * K}
    if kind == "rows":
        n = c["rows"] * c["K"]
        return {"bytes": 3 * n + n // BLOCK * 4, "flops": 2 * n}
    if kind == "weight":
        n, times = c["G"] * c["N"] * c["K"], 2 if c["t"] else 1
        return {"bytes": n * (4 if c["w"] == "f32" else 2) + times * (n + n // BLOCK ** 2 * 4), "flops": 2 * n}
    sizes = _tensor_sizes(c["tensors"], c["elements"])
    bound = sorted(sizes)[len(sizes) // 2]
    once = sum(n * (4 if n >= bound else 2) for n in sizes)
    # the norm has to be known before the first value can be scaled: two reads and a write, or one read
    return {"bytes": once * (3 if c["clipped"] else 1), "flops": sum(sizes) * (3 if c["clipped"] else 2)}


# ---------------------------------------------------------------- the definitions, in 64 bits

def _codes64(v, amax):
    """e4m3 values of v / (amax / 448): the nearest multiple of the binade's step, ties to the even one."""
    sc = torch.where(amax > 0, amax / E4M3_MAX, torch.ones_like(amax))
    q = (v / sc).clamp(-E4M3_MAX, E4M3_MAX)
    step = torch.exp2(torch.frexp(q.abs().clamp_min(2.0 ** -6)).exponent.double() - 4.0)
    return torch.round(q / step) * step, sc


def exact(case, seed):
    c, kind = case, case["kind"]
    s = prepare(case, seed)
    if kind in ("fwd", "dgrad", "wgrad"):
        G, M, N, K = c["G"], c["M"], c["N"], c["K"]
        shape = {"fwd": (M, N), "dgrad": (M, K), "wgrad": (G, N, K)}[kind]
        out = torch.zeros(shape, dtype=torch.float64, device="cuda")
        at = 0
        for e, m in enumerate(s["rows"]):
            r = slice(at, at + m)
            at += m
            if kind == "fwd":
                torch.matmul(s["x"][r].double(), s["w"][e].double().t(), out=out[r])
            elif kind == "dgrad":
                torch.matmul(s["dy"][r].double(), s["w"][e].double(), out=out[r])
            elif m:
                torch.matmul(s["dy"][r].double().t(), s["x"][r].double(), out=out[e])
        return out
    if kind == "rows":
        b = s["x"].double().view(c["rows"], -1, BLOCK)
        q, sc = _codes64(b, b.abs().amax(-1, keepdim=True))
        return {"codes": q.view(c["rows"], c["K"]), "scale": sc[..., 0]}
    if kind == "weight":
        q = torch.empty(s["w"].shape, dtype=torch.float64, device="cuda")
        sc = torch.empty(c["G"], c["N"] // BLOCK, c["K"] // BLOCK, dtype=torch.float64, device="cuda")
        for e, w in enumerate(s["w"]):
            for i, rows in enumerate(w.double().split(BLOCK, 0)):
                b = rows.view(BLOCK, -1, BLOCK)
                codes, scale = _codes64(b, b.abs().amax(2, keepdim=True).amax(0, keepdim=True))
                q[e, i * BLOCK:(i + 1) * BLOCK] = codes.view(BLOCK, c["K"])
                sc[e, i] = scale.flatten()
        return {"codes": q, "scale": sc, **({"codes_t": q.mT.contiguous(), "scale_t": sc.mT.contiguous()} if c["t"] else {})}
    total = math.fsum(float(part.double().pow(2).sum()) for flat in s["flat"] for part in flat.split(1 << 26))
    norm = math.sqrt(total)
    factor = min(1.0, s["max_norm"] / (norm + 1e-6))
    return {"norm": torch.tensor([norm], dtype=torch.float64, device="cuda"), "f32": s["flat"][0].double() * factor,
            "bf16": s["flat"][1].double() * factor}
