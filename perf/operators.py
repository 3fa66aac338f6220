"""Cases that measure the operators around the grouped GEMM in a mixture-of-experts layer.

    normalise      f8f8bf16_rmsnorm_quantize, f8f8bf16_rmsnorm_backward
    route          f8f8bf16_route, f8f8bf16_route_backward
    exchange       f8f8bf16_moe_dispatch, f8f8bf16_moe_combine, f8f8bf16_moe_combine_backward
    checkpoint     f8f8bf16_silu_mul_quantize, f8f8bf16_silu_mul_backward, f8f8bf16_quantize_k_offsets

With ``own`` false ``run`` computes an operator from elementary torch operations,
with ``own`` true it makes the library's call.  Sizes: the hidden size 7168, the
expert sizes N = 4096 (gate and up, 2048 each) and K = 7184, N = 1000 tails are
those of the grouped GEMM workloads of this repository; the others are generic.
"""
import math

import torch

own = False

E4M3_MAX = 448.0
FP8 = torch.float8_e4m3fn
BLOCK = 128


def listed():
    return [
        # one decode step of eight sequences: the norm before the experts, residual added, codes for the gate_up product
        {"name": "norm_decode", "kind": "norm", "rows": 8, "K": 7168, "residual": True, "block": 0, "y": False, "w": "bf16"},
        # a long prompt: block scales for the block-scaled products, the bf16 rows too for the router's own product
        {"name": "norm_prefill_blocks", "kind": "norm", "rows": 16384, "K": 7168, "residual": True, "block": 128, "y": True, "w": "bf16"},
        # training, an odd number of rows, K with a tail, fp32 weights, the residual stream's gradient added
        {"name": "norm_backward", "kind": "norm_bwd", "rows": 4093, "K": 7184, "dres": True, "w": "f32"},
        # one decode step of sixteen sequences over eight experts, two each
        {"name": "route_decode", "kind": "route", "T": 16, "E": 8, "k": 2, "score": "softmax", "bias": False, "n_group": 1,
         "topk_group": 1, "group_top": 1, "renorm": True, "scale": 1.0, "dtype": "f32"},
        # a long prompt over 256 experts in eight groups, four of them kept, a balancing bias
        {"name": "route_prefill_groups", "kind": "route", "T": 16384, "E": 256, "k": 8, "score": "sigmoid", "bias": True, "n_group": 8,
         "topk_group": 4, "group_top": 2, "renorm": True, "scale": 2.5, "dtype": "f32"},
        # training: the gradient of bf16 logits, an odd number of tokens
        {"name": "route_backward", "kind": "route_bwd", "T": 8191, "E": 128, "k": 8, "score": "softmax", "renorm": True, "scale": 1.0,
         "dtype": "bf16"},
        # a decode step's codes and scales copied into the experts' order
        {"name": "dispatch_decode", "kind": "dispatch", "T": 64, "E": 32, "k": 8, "K": 7168, "block": 0},
        # a prompt's expert outputs summed back per token, a shared expert's output added
        {"name": "combine_prefill", "kind": "combine", "T": 4096, "E": 32, "k": 8, "N": 7168, "addend": True},
        # training: the gradients of the expert outputs and of the routing weights, an odd number of tokens
        {"name": "combine_backward", "kind": "combine_bwd", "T": 2047, "E": 32, "k": 8, "N": 7168},
        # training forward: the gated activation's codes for the down product and the 8-bit checkpoint of its input
        {"name": "act_checkpoint", "kind": "act", "rows": 16384, "I": 2048, "block": 0, "ckpt": True},
        # training backward from the 8-bit checkpoint, odd rows, a last block cut short
        {"name": "act_backward_tail", "kind": "act_bwd", "rows": 5001, "I": 1000},
        # the weight gradient's operand, from the 8-bit activations that the forward pass kept
        {"name": "wgrad_operand", "kind": "wgrad", "R": 4096, "G": 8, "K": 7168, "src": "fp8", "block": 0},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    """One more case: sizes over the logarithm of their range, odd rows, widths in whole store granules."""
    kind = rng.choice(["norm", "norm_bwd", "route", "route_bwd", "dispatch", "combine", "combine_bwd", "act", "act_bwd", "wgrad"])
    most = 100_000_000                       # elements, about the largest listed case
    if kind in ("norm", "norm_bwd"):
        K = 8 * _log(rng, 32, 1280)
        block = rng.choice([0, 128]) if kind == "norm" else 0
        K = max(128, K // 128 * 128) if block else K
        rows = min(_log(rng, 1, 20000), most // K)
        if kind == "norm":
            return {"kind": kind, "rows": rows, "K": K, "residual": rng.random() < 0.7, "block": block, "y": rng.random() < 0.4,
                    "w": rng.choice(["bf16", "f32"])}
        return {"kind": kind, "rows": rows, "K": K, "dres": rng.random() < 0.7, "w": rng.choice(["bf16", "f32"])}
    if kind in ("route", "route_bwd"):
        n_group = rng.choice([1, 1, 4, 8]) if kind == "route" else 1
        E = n_group * _log(rng, 8 if n_group == 1 else 4, 384 // n_group)
        k = min(rng.choice([1, 2, 4, 6, 8]), E)
        topk_group = rng.randint(max(1, n_group // 2), n_group)
        k = min(k, topk_group * (E // n_group))
        T = min(_log(rng, 1, 24000), 5_000_000 // E)
        score, scale = rng.choice(["softmax", "sigmoid"]), rng.choice([1.0, 2.5])
        dtype = rng.choice(["f32", "bf16"])
        if kind == "route":
            return {"kind": kind, "T": T, "E": E, "k": k, "score": score, "bias": rng.random() < 0.5, "n_group": n_group,
                    "topk_group": topk_group, "group_top": rng.choice([1, 2]) if n_group > 1 else 1, "renorm": rng.random() < 0.7,
                    "scale": scale, "dtype": dtype}
        return {"kind": kind, "T": T, "E": E, "k": k, "score": score, "renorm": rng.random() < 0.7, "scale": scale, "dtype": dtype}
    if kind in ("dispatch", "combine", "combine_bwd"):
        E = _log(rng, 8, 256)
        k = min(rng.choice([1, 2, 4, 6, 8]), E)
        block = rng.choice([0, 128]) if kind == "dispatch" else 0
        N = 16 * _log(rng, 16, 512)
        N = max(128, N // 128 * 128) if block else N
        T = max(1, min(_log(rng, 1, 8000), 2 * most // (N * k)))
        if kind == "dispatch":
            return {"kind": kind, "T": T, "E": E, "k": k, "K": N, "block": block}
        if kind == "combine":
            return {"kind": kind, "T": T, "E": E, "k": k, "N": N, "addend": rng.random() < 0.5}
        return {"kind": kind, "T": T, "E": E, "k": k, "N": N}
    if kind in ("act", "act_bwd"):
        I = 8 * _log(rng, 16, 1024)
        block = rng.choice([0, 128]) if kind == "act" else 0
        I = max(128, I // 128 * 128) if block else I
        rows = min(_log(rng, 1, 32000), most // (2 * I))
        if kind == "act":
            return {"kind": kind, "rows": rows, "I": I, "block": block, "ckpt": rng.random() < 0.6}
        return {"kind": kind, "rows": rows, "I": I}
    K = 16 * _log(rng, 16, 512)
    src = rng.choice(["fp8", "bf16"])
    block = rng.choice([0, 128]) if src == "fp8" else 0
    K = max(128, K // 128 * 128) if block else K
    return {"kind": kind, "R": min(_log(rng, 1, 20000), most // (2 * K)), "G": _log(rng, 1, 64), "K": K, "src": src, "block": block}


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


def _weight(g, K, w):
    v = 1.0 + 0.2 * _normal(g, K)
    return v if w == "f32" else v.to(torch.bfloat16)


def _quantized(g, rows, K, block):
    """Codes and scales as the library's quantisers leave them."""
    x = _acts(g, rows, K).float()
    b = x.view(rows, K // BLOCK, BLOCK) if block else x.view(rows, 1, K)
    s = b.abs().amax(-1) / E4M3_MAX
    s = torch.where(s > 0, s, torch.ones_like(s))
    q = (b / s.unsqueeze(-1)).clamp(-E4M3_MAX, E4M3_MAX).to(FP8).view(rows, K)
    return q.view(torch.uint8), (s if block else s.view(rows))


def _routing(g, T, E, k):
    """A skewed routing: distinct experts per token, positions in the experts' order."""
    score = _normal(g, T, E) + 0.5 * _normal(g, 1, E)
    ids = score.topk(k, dim=1).indices
    order = torch.sort(ids.reshape(-1), stable=True).indices
    dst = torch.empty(T * k, dtype=torch.int32, device="cuda")
    dst[order] = torch.arange(T * k, dtype=torch.int32, device="cuda")
    w = torch.rand(T, k, generator=g, device="cuda") + 0.05
    return ids.to(torch.int32), dst.view(T, k), w / w.sum(1, keepdim=True)


def _sizes(g, G, R):
    """Rows per expert: skewed, an expert now and then empty."""
    p = torch.exp(_normal(g, G)) * (torch.rand(G, generator=g, device="cuda") > 0.1)
    p[0] += 1e-3
    cut = (torch.cumsum(p / p.sum(), 0) * R).round().to(torch.int64)
    cut[-1] = R
    return torch.diff(cut, prepend=cut.new_zeros(1))


def prepare(case, seed):
    g, c, kind = _gen(seed), dict(case), case["kind"]
    s = {"case": c}
    if kind == "norm":
        s["x"] = _acts(g, c["rows"], c["K"])
        s["residual"] = _acts(g, c["rows"], c["K"]) if c["residual"] else None
        s["weight"] = _weight(g, c["K"], c["w"])
    elif kind == "norm_bwd":
        s["h"] = _acts(g, c["rows"], c["K"])
        s["rstd"] = torch.rsqrt(s["h"].double().square().mean(1) + 1e-6).float()
        s["weight"] = _weight(g, c["K"], c["w"])
        s["dy"] = _normal(g, c["rows"], c["K"], sigma=1e-2).to(torch.bfloat16)
        s["dres"] = _normal(g, c["rows"], c["K"], sigma=1e-2).to(torch.bfloat16) if c["dres"] else None
    elif kind in ("route", "route_bwd"):
        x = _normal(g, c["T"], c["E"], sigma=1.5) + 0.3 * _normal(g, 1, c["E"])
        s["logits"] = x if c["dtype"] == "f32" else x.to(torch.bfloat16)
        if kind == "route":
            s["bias"] = 0.05 * _normal(g, c["E"]) if c["bias"] else None
        else:
            s["ids"] = x.topk(c["k"], dim=1).indices.to(torch.int32)
            s["dw"] = _normal(g, c["T"], c["k"])
    elif kind in ("dispatch", "combine", "combine_bwd"):
        _, s["dst"], s["w"] = _routing(g, c["T"], c["E"], c["k"])
        if kind == "dispatch":
            s["xq"], s["xs"] = _quantized(g, c["T"], c["K"], c["block"])
        else:
            s["y"] = _acts(g, c["T"] * c["k"], c["N"])
            if kind == "combine":
                s["addend"] = _acts(g, c["T"], c["N"]) if c["addend"] else None
            else:
                s["dout"] = _normal(g, c["T"], c["N"], sigma=1e-2).to(torch.bfloat16)
    elif kind == "act":
        s["h"] = _acts(g, c["rows"], 2 * c["I"])
    elif kind == "act_bwd":
        rows, I = c["rows"], c["I"]
        nb = -(-I // BLOCK)
        h = torch.zeros(rows, 2, nb * BLOCK, device="cuda")
        h[:, :, :I] = _acts(g, rows, 2 * I).float().view(rows, 2, I)
        b = h.view(rows, 2, nb, BLOCK)
        sc = b.abs().amax(-1) / E4M3_MAX
        s["h_scale"] = torch.where(sc > 0, sc, torch.ones_like(sc))
        q = (b / s["h_scale"].unsqueeze(-1)).clamp(-E4M3_MAX, E4M3_MAX).view(rows, 2, nb * BLOCK)[:, :, :I]
        s["hq"] = q.to(FP8).view(torch.uint8).reshape(rows, 2 * I)
        s["da"] = _normal(g, rows, I, sigma=1e-2).to(torch.bfloat16)
    else:
        s["sizes"] = _sizes(g, c["G"], c["R"])
        if c["src"] == "fp8":
            s["x"], s["xs"] = _quantized(g, c["R"], c["K"], c["block"])
        else:
            s["x"], s["xs"] = _normal(g, c["R"], c["K"], sigma=1e-2).to(torch.bfloat16), None
    return s


# ---------------------------------------------------------------- one pass

def run(state):
    if own:
        import fp8_rowwise_scaled_amd as F
        return _OWN[state["case"]["kind"]](F, state, state["case"])
    return _PLAIN[state["case"]["kind"]](state, state["case"])


def _own_norm(F, s, c):
    r = F.f8f8bf16_rmsnorm_quantize(s["x"], s["weight"], 1e-6, residual=s["residual"], block=c["block"], want_y=c["y"], want_rstd=True)
    return {"codes": r.XQ.view(FP8), "scale": r.x_scale, "rstd": r.rstd, **({"residual": r.residual} if c["residual"] else {}),
            **({"y": r.Y} if c["y"] else {})}


def _own_norm_bwd(F, s, c):
    dx, dw = F.f8f8bf16_rmsnorm_backward(s["dy"], s["h"], s["weight"], s["rstd"], dresidual=s["dres"])
    return {"dx": dx, "dw": dw}


def _own_route(F, s, c):
    r = F.f8f8bf16_route(s["logits"], c["k"], bias=s["bias"], score=c["score"], n_group=c["n_group"], topk_group=c["topk_group"],
                         group_top=c["group_top"], renormalize=c["renorm"], scale=c["scale"])
    return {"weights": r.weights, "ids": r.ids, "sizes": r.M_sizes, "dst": r.dst_row}


def _own_route_bwd(F, s, c):
    return F.f8f8bf16_route_backward(s["logits"], s["ids"], s["dw"], score=c["score"], renormalize=c["renorm"], scale=c["scale"])


def _own_dispatch(F, s, c):
    q, sc = F.f8f8bf16_moe_dispatch(s["xq"], s["xs"], s["dst"])
    return {"codes": q.view(FP8), "scale": sc}


def _own_combine(F, s, c):
    return F.f8f8bf16_moe_combine(s["y"], s["dst"], s["w"], addend=s["addend"])


def _own_combine_bwd(F, s, c):
    dy, dw = F.f8f8bf16_moe_combine_backward(s["dout"], s["dst"], s["w"], s["y"])
    return {"dy": dy, "dw": dw}


def _own_act(F, s, c):
    r = F.f8f8bf16_silu_mul_quantize(s["h"], block=c["block"], checkpoint=c["ckpt"])
    return {"codes": r.AQ.view(FP8), "scale": r.a_scale, **({"hq": r.HQ.view(FP8), "h_scale": r.h_scale} if c["ckpt"] else {})}


def _own_act_bwd(F, s, c):
    return F.f8f8bf16_silu_mul_backward(s["da"], s["hq"], s["h_scale"])


def _own_wgrad(F, s, c):
    xt, ts, ko = F.f8f8bf16_quantize_k_offsets(s["x"], s["sizes"], x_scale=s["xs"])
    return {"codes": xt.view(FP8), "scale": ts, "k_offsets": ko}


_OWN = {"norm": _own_norm, "norm_bwd": _own_norm_bwd, "route": _own_route, "route_bwd": _own_route_bwd, "dispatch": _own_dispatch,
        "combine": _own_combine, "combine_bwd": _own_combine_bwd, "act": _own_act, "act_bwd": _own_act_bwd, "wgrad": _own_wgrad}


def _to_codes(v, s):
    return (v / s).clamp(-E4M3_MAX, E4M3_MAX).to(FP8)


def _scale_of(amax):
    return torch.where(amax > 0, amax / E4M3_MAX, 1.0)


def _plain_quantize(v, block):
    rows, K = v.shape
    if not block:
        s = _scale_of(v.abs().amax(1, keepdim=True))
        return _to_codes(v, s), s.view(rows)
    b = v.view(rows, K // BLOCK, BLOCK)
    s = _scale_of(b.abs().amax(-1, keepdim=True))
    return _to_codes(b, s).view(rows, K), s.view(rows, K // BLOCK)


def _plain_norm(s, c):
    h = s["x"]
    if c["residual"]:
        h = (h.float() + s["residual"].float()).to(torch.bfloat16)
    hf = h.float()
    rstd = torch.rsqrt((hf * hf).mean(1) + 1e-6)
    y = hf * rstd[:, None] * s["weight"].float()
    q, sc = _plain_quantize(y, c["block"])
    return {"codes": q, "scale": sc, "rstd": rstd, **({"residual": h} if c["residual"] else {}),
            **({"y": y.to(torch.bfloat16)} if c["y"] else {})}


def _plain_norm_bwd(s, c):
    r, dy = s["rstd"][:, None], s["dy"].float()
    xhat = s["h"].float() * r
    wdy = dy * s["weight"].float()
    dx = r * (wdy - xhat * (wdy * xhat).mean(1, keepdim=True))
    if c["dres"]:
        dx = dx + s["dres"].float()
    return {"dx": dx.to(torch.bfloat16), "dw": (dy * xhat).sum(0)}


def _plain_scores(x, score):
    if score == "sigmoid":
        return 1.0 / (1.0 + torch.exp(-x))
    e = torch.exp(x - x.amax(1, keepdim=True))
    return e / e.sum(1, keepdim=True)


def _plain_route(s, c):
    x = s["logits"].float()
    T, E, k = c["T"], c["E"], c["k"]
    # The order of bare scores is that of the logits; sums with a bias, or of two scores, are compared in 64 bits.
    if c["bias"] or (c["n_group"] > 1 and c["group_top"] == 2):
        key = _plain_scores(x.double(), c["score"])
        key = key + s["bias"].double() if c["bias"] else key
    else:
        key = x
    if c["n_group"] > 1:
        grouped = key.view(T, c["n_group"], -1)
        gs = grouped.amax(-1) if c["group_top"] == 1 else grouped.topk(min(2, E // c["n_group"]), dim=-1).values.sum(-1)
        kept = torch.sort(gs, dim=1, descending=True, stable=True).indices[:, :c["topk_group"]]
        mask = torch.zeros_like(gs, dtype=torch.bool).scatter_(1, kept, True)
        key = grouped.masked_fill(~mask[:, :, None], float("-inf")).view(T, E)
    ids = torch.sort(key, dim=1, descending=True, stable=True).indices[:, :k]
    w = _plain_scores(x, c["score"]).gather(1, ids)
    if c["renorm"]:
        w = w / (w.sum(1, keepdim=True) + 1e-20)
    flat = ids.reshape(-1)
    sizes = torch.zeros(E, dtype=torch.int64, device=x.device).scatter_add_(0, flat, torch.ones_like(flat))
    order = torch.sort(flat, stable=True).indices
    dst = torch.empty(T * k, dtype=torch.int32, device=x.device)
    dst[order] = torch.arange(T * k, dtype=torch.int32, device=x.device)
    return {"weights": w * c["scale"], "ids": ids.to(torch.int32), "sizes": sizes, "dst": dst.view(T, k)}


def _plain_route_bwd(s, c):
    x, ids = s["logits"].float(), s["ids"].long()
    dw = s["dw"] * c["scale"]
    p = _plain_scores(x, c["score"])
    ps = p.gather(1, ids)
    if c["renorm"]:
        total = ps.sum(1, keepdim=True) + 1e-20
        dps = (dw - (dw * ps).sum(1, keepdim=True) / total) / total
    else:
        dps = dw
    dp = torch.zeros_like(x).scatter_(1, ids, dps)
    if c["score"] == "sigmoid":
        dx = dp * p * (1.0 - p)
    else:
        dx = p * (dp - (dp * p).sum(1, keepdim=True))
    return dx.to(s["logits"].dtype)


def _plain_dispatch(s, c):
    flat = s["dst"].reshape(-1).long()
    src = torch.empty_like(flat)
    src[flat] = torch.arange(flat.numel(), device=flat.device)
    src = src // c["k"]
    return {"codes": s["xq"][src].view(FP8), "scale": s["xs"][src]}


def _plain_combine(s, c):
    out = (s["y"][s["dst"].long()].float() * s["w"][:, :, None]).sum(1)
    if c["addend"]:
        out = out + s["addend"].float()
    return out.to(torch.bfloat16)


def _plain_combine_bwd(s, c):
    d, dst = s["dout"].float(), s["dst"].long()
    dw = (s["y"][dst].float() * d[:, None, :]).sum(-1)
    dy = torch.empty_like(s["y"])
    dy[dst.reshape(-1)] = (d[:, None, :] * s["w"][:, :, None]).to(torch.bfloat16).view(-1, c["N"])
    return {"dy": dy, "dw": dw}


def _plain_act(s, c):
    rows, I = c["rows"], c["I"]
    h = s["h"].float()
    gate, up = h[:, :I], h[:, I:]
    q, sc = _plain_quantize(gate / (1.0 + torch.exp(-gate)) * up, c["block"])
    out = {"codes": q, "scale": sc}
    if c["ckpt"]:
        nb = -(-I // BLOCK)
        b = torch.nn.functional.pad(h.view(rows, 2, I), (0, nb * BLOCK - I)).view(rows, 2, nb, BLOCK)
        hs = _scale_of(b.abs().amax(-1, keepdim=True))
        out["hq"] = _to_codes(b, hs).view(rows, 2, nb * BLOCK)[:, :, :I].reshape(rows, 2 * I)
        out["h_scale"] = hs.view(rows, 2, nb)
    return out


def _plain_act_bwd(s, c):
    rows, I = c["rows"], c["I"]
    sc = s["h_scale"].repeat_interleave(BLOCK, dim=2)[:, :, :I]
    h = s["hq"].view(FP8).float().view(rows, 2, I) * sc
    gate, up, da = h[:, 0], h[:, 1], s["da"].float()
    sig = 1.0 / (1.0 + torch.exp(-gate))
    return torch.cat([da * up * sig * (1.0 + gate * (1.0 - sig)), da * gate * sig], 1).to(torch.bfloat16)


def _plain_wgrad(s, c):
    R, G, K = c["R"], c["G"], c["K"]
    if c["src"] == "fp8":
        v = s["x"].view(FP8).float()
        v = (v.view(R, K // BLOCK, BLOCK) * s["xs"][:, :, None]).view(R, K) if c["block"] else v * s["xs"][:, None]
    else:
        v = s["x"].float()
    ends = torch.cumsum(s["sizes"], 0)
    group = torch.searchsorted(ends, torch.arange(R, device=v.device), right=True)
    amax = torch.segment_reduce(v.abs(), "max", lengths=s["sizes"], axis=0, initial=0.0, unsafe=True)
    sc = _scale_of(amax)
    padded = torch.cumsum((s["sizes"] + 15) // 16 * 16, 0)
    at = torch.arange(R, device=v.device) + (padded - ends - (s["sizes"] + 15) // 16 * 16 + s["sizes"])[group]
    out = torch.zeros(K, _capacity(R, G), dtype=torch.uint8, device=v.device)
    out[:, at] = _to_codes(v, sc[group]).view(torch.uint8).t()
    return {"codes": out.view(FP8), "scale": sc, "k_offsets": padded.to(torch.int32)}


_PLAIN = {"norm": _plain_norm, "norm_bwd": _plain_norm_bwd, "route": _plain_route, "route_bwd": _plain_route_bwd,
          "dispatch": _plain_dispatch, "combine": _plain_combine, "combine_bwd": _plain_combine_bwd, "act": _plain_act,
          "act_bwd": _plain_act_bwd, "wgrad": _plain_wgrad}


def _capacity(R, G):
    """Columns of the weight gradient's operand: every group's rows rounded up to 16."""
    return -(-(R + 15 * min(R, G)) // 16) * 16


# ---------------------------------------------------------------- what a pass cannot do without

def work(case):
    c, kind = case, case["kind"]
    if kind == "norm":
        n, sc = c["rows"] * c["K"], c["rows"] * (c["K"] // BLOCK if c["block"] else 1)
        return {"bytes": n * (2 + (4 if c["residual"] else 0) + 1 + (2 if c["y"] else 0)) + c["K"] * (4 if c["w"] == "f32" else 2)
                + 4 * sc + 4 * c["rows"], "flops": 8 * n}
    if kind == "norm_bwd":
        n = c["rows"] * c["K"]
        return {"bytes": n * (6 + (2 if c["dres"] else 0)) + c["K"] * (8 if c["w"] == "f32" else 6) + 4 * c["rows"], "flops": 11 * n}
    if kind == "route":
        n, m = c["T"] * c["E"], c["T"] * c["k"]
        return {"bytes": n * (4 if c["dtype"] == "f32" else 2) + (4 * c["E"] if c["bias"] else 0) + 12 * m + 8 * c["E"], "flops": n * 6}
    if kind == "route_bwd":
        n, m, e = c["T"] * c["E"], c["T"] * c["k"], 4 if c["dtype"] == "f32" else 2
        every = c["score"] == "softmax" and not c["renorm"]     # else only the chosen logits matter
        return {"bytes": n * e + (n if every else m) * e + 8 * m, "flops": (n if every else m) * 10}
    if kind == "dispatch":
        row = c["K"] + 4 * (c["K"] // BLOCK if c["block"] else 1)
        return {"bytes": c["T"] * row * (1 + c["k"]) + 4 * c["T"] * c["k"], "flops": 0}
    if kind == "combine":
        n = c["T"] * c["N"]
        return {"bytes": n * 2 * (c["k"] + 1 + (1 if c["addend"] else 0)) + 8 * c["T"] * c["k"], "flops": 2 * n * c["k"]}
    if kind == "combine_bwd":
        n = c["T"] * c["N"]
        return {"bytes": n * 2 * (1 + 2 * c["k"]) + 12 * c["T"] * c["k"], "flops": 3 * n * c["k"]}
    nb = -(-c["I"] // BLOCK) if "I" in c else 0
    if kind == "act":
        n = c["rows"] * c["I"]
        sc = c["rows"] * (c["I"] // BLOCK if c["block"] else 1)
        return {"bytes": n * (5 + (2 if c["ckpt"] else 0)) + 4 * sc + (8 * c["rows"] * nb if c["ckpt"] else 0), "flops": 10 * n}
    if kind == "act_bwd":
        n = c["rows"] * c["I"]
        return {"bytes": n * 8 + 8 * c["rows"] * nb, "flops": 14 * n}
    n = c["R"] * c["K"]
    sc = (c["R"] * (c["K"] // BLOCK if c["block"] else 1) * 4) if c["src"] == "fp8" else 0
    return {"bytes": n * (1 if c["src"] == "fp8" else 2) + c["K"] * _capacity(c["R"], c["G"]) + sc + c["G"] * (12 + 4 * c["K"]),
            "flops": 4 * n}


# ---------------------------------------------------------------- the definitions, in 64 bits

def _codes64(v, amax):
    """e4m3 values of v / (amax / 448): the nearest multiple of the binade's step, ties to the even one."""
    s = torch.where(amax > 0, amax / E4M3_MAX, torch.ones_like(amax))
    q = (v / s).clamp(-E4M3_MAX, E4M3_MAX)
    e = torch.frexp(q.abs().clamp_min(2.0 ** -6)).exponent.double() - 1.0
    step = torch.exp2(e - 3.0)
    return torch.round(q / step) * step, s


def _blocks64(v, block):
    rows, K = v.shape
    b = v.reshape(rows, -1, block if block else K)
    q, s = _codes64(b, b.abs().amax(-1, keepdim=True))
    return q.reshape(rows, K), (s.reshape(rows, -1) if block else s.reshape(rows))


def _scores64(x, score):
    return torch.sigmoid(x) if score == "sigmoid" else torch.softmax(x, 1)


def exact(case, seed):
    c, kind = case, case["kind"]
    s = prepare(case, seed)
    if kind == "norm":
        h = s["x"].double()
        if c["residual"]:
            h = (h + s["residual"].double()).float().to(torch.bfloat16).double()    # a bf16 sum is exact in fp32 or rounds the same
        rstd = 1.0 / torch.sqrt(h.pow(2).mean(1) + 1e-6)
        y = h * s["weight"].double() * rstd[:, None]
        q, sc = _blocks64(y, c["block"])
        return {"codes": q, "scale": sc, "rstd": rstd, **({"residual": h} if c["residual"] else {}), **({"y": y} if c["y"] else {})}
    if kind == "norm_bwd":
        h, dy, r, w = s["h"].double(), s["dy"].double(), s["rstd"].double()[:, None], s["weight"].double()
        dot = (h * dy * w).sum(1, keepdim=True)
        dx = r * w * dy - r ** 3 * h * dot / c["K"]
        return {"dx": dx + s["dres"].double() if c["dres"] else dx, "dw": (dy * h * r).sum(0)}
    if kind == "route":
        x = s["logits"].double()
        p = _scores64(x, c["score"])
        key = p + s["bias"].double() if c["bias"] else x if c["n_group"] == 1 or c["group_top"] == 1 else p
        if c["n_group"] > 1:
            per = c["E"] // c["n_group"]
            top = torch.sort(key.view(c["T"], c["n_group"], per), dim=-1, descending=True).values
            gs = top[..., :c["group_top"]].sum(-1)
            at = torch.argsort(torch.argsort(gs, dim=1, descending=True, stable=True), dim=1)
            key = torch.where((at < c["topk_group"]).repeat_interleave(per, 1), key, torch.full_like(key, -math.inf))
        ids = torch.argsort(key, dim=1, descending=True, stable=True)[:, :c["k"]]
        w = torch.take_along_dim(p, ids, 1)
        w = w / w.sum(1, keepdim=True) if c["renorm"] else w
        order = torch.argsort(ids.flatten(), stable=True)
        return {"weights": w * c["scale"], "ids": ids.to(torch.int32), "sizes": torch.bincount(ids.flatten(), minlength=c["E"]),
                "dst": torch.argsort(order).to(torch.int32).view(c["T"], c["k"])}
    if kind == "route_bwd":
        x = s["logits"].double().requires_grad_(True)
        w = torch.take_along_dim(_scores64(x, c["score"]), s["ids"].long(), 1)
        w = w / w.sum(1, keepdim=True) if c["renorm"] else w
        return torch.autograd.grad((w * c["scale"] * s["dw"].double()).sum(), x)[0]
    if kind == "dispatch":
        token = torch.argsort(s["dst"].flatten().long()) // c["k"]
        return {"codes": s["xq"].view(FP8).double()[token], "scale": s["xs"].double()[token]}
    if kind == "combine":
        out = torch.bmm(s["w"].double()[:, None, :], s["y"].double()[s["dst"].long()])[:, 0]
        return out + s["addend"].double() if c["addend"] else out
    if kind == "combine_bwd":
        token = torch.argsort(s["dst"].flatten().long())
        d = s["dout"].double()
        dw = torch.bmm(s["y"].double()[s["dst"].long()], d[:, :, None])[:, :, 0]
        return {"dy": d[token // c["k"]] * s["w"].double().flatten()[token][:, None], "dw": dw}
    if kind == "act":
        gate, up = s["h"].double().chunk(2, 1)
        q, sc = _blocks64(gate * torch.sigmoid(gate) * up, c["block"])
        out = {"codes": q, "scale": sc}
        if c["ckpt"]:
            halves = [[_codes64(b, b.abs().amax(1, keepdim=True)) for b in half.split(BLOCK, 1)] for half in (gate, up)]
            out["hq"] = torch.cat([q for half in halves for q, _ in half], 1)
            out["h_scale"] = torch.stack([torch.cat([sc for _, sc in half], 1) for half in halves], 1)
        return out
    if kind == "act_bwd":
        nb = s["h_scale"].shape[2]
        block = torch.arange(c["I"], device="cuda") // BLOCK
        hq = s["hq"].view(FP8).double()
        gate = (hq[:, :c["I"]] * s["h_scale"][:, 0].double()[:, block]).requires_grad_(True)
        up = (hq[:, c["I"]:] * s["h_scale"][:, 1].double()[:, block]).requires_grad_(True)
        assert nb == block[-1] + 1
        dg, du = torch.autograd.grad(torch.nn.functional.silu(gate) * up, (gate, up), s["da"].double())
        return torch.cat([dg, du], 1)
    v = s["x"].view(FP8).double() if c["src"] == "fp8" else s["x"].double()
    if c["src"] == "fp8":
        v = v * (s["xs"].double().repeat_interleave(BLOCK, 1) if c["block"] else s["xs"].double()[:, None])
    codes = torch.zeros(c["K"], _capacity(c["R"], c["G"]), dtype=torch.float64, device="cuda")
    scales, ends, row, col = [], [], 0, 0
    for m in s["sizes"].tolist():
        part = v[row:row + m]
        amax = part.abs().amax(0) if m else torch.zeros(c["K"], dtype=torch.float64, device="cuda")
        q, sc = _codes64(part, amax[None])
        codes[:, col:col + m] = q.t()
        row, col = row + m, col + -(-m // 16) * 16
        scales.append(sc[0])
        ends.append(col)
    return {"codes": codes, "scale": torch.stack(scales), "k_offsets": torch.tensor(ends, dtype=torch.int32, device="cuda")}
