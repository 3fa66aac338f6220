"""One mixture-of-experts layer from this library's operators: forward, and a training
step's backward pass.

    python examples/moe_layer.py [--tokens T --hidden H --inner I --experts E --topk K] [--steps N]

Forward:   norm with fp8 output -> router -> rows to the experts -> gate and up product
           -> gated activation with fp8 output and 8-bit checkpoint -> down product
           -> weighted sum back to the tokens, plus the residual stream.
Backward:  from the gradient of the layer's output to those of its input, of the norm's
           and the router's weights and of both expert weights.  What the forward pass
           keeps of the activations is in 8 bits: the fp8 rows that the products read and
           the checkpoint of the gated activation's input.

Training:  ``train_step`` keeps fp32 weights, quantises them for the block-scaled products
           of both passes (or uses bf16 products instead), adds the weights' gradients up in
           fp32 over micro-batches with bf16 products, clips them by their common norm, and
           updates the weights.  With bf16 products nothing is in 8 bits: the gated activation
           between them and its gradient are then torch's, from the bf16 rows kept.

The router's own product (tokens x hidden x experts, small) is torch's.  ``main`` runs the
layer on random data, compares it with the same layer in fp32 torch operations, and
times both passes and a training step.
"""
from __future__ import annotations

import argparse
import os
import sys
import time
from dataclasses import dataclass

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import fp8_rowwise_scaled_amd as F  # noqa: E402


def quantize_weight(w: torch.Tensor):
    """[G, N, K] float -> fp8 codes and one scale per output column."""
    G, N, K = w.shape
    q, s = F.f8f8bf16_quantize_rowwise(w.to(torch.bfloat16).reshape(G * N, K).contiguous())
    return q.view(G, N, K), s.view(G, N)


@dataclass
class Weights:
    norm: torch.Tensor        # [H] float32
    router: torch.Tensor      # [E, H] float32
    bias: torch.Tensor        # [E] float32, for the choice only
    w1: torch.Tensor          # [E, 2 I, H] float32: gate and up
    w2: torch.Tensor          # [E, H, I] float32: down

    def quantized(self):
        """The products' operands, laid out once: both weights and their transposes."""
        return {"w1": quantize_weight(self.w1), "w2": quantize_weight(self.w2),
                "w1t": quantize_weight(self.w1.transpose(1, 2)), "w2t": quantize_weight(self.w2.transpose(1, 2))}


def random_weights(H: int, I: int, E: int, seed: int = 0, device: str = "cuda") -> Weights:
    g = torch.Generator(device=device).manual_seed(seed)

    def normal(*shape, sigma):
        return torch.randn(*shape, generator=g, device=device) * sigma
    return Weights(1 + normal(H, sigma=0.1), normal(E, H, sigma=H ** -0.5), normal(E, sigma=0.01),
                   normal(E, 2 * I, H, sigma=H ** -0.5), normal(E, H, I, sigma=I ** -0.5))


def forward(x, residual, w: Weights, q: dict, k: int):
    """(output, residual stream, what the backward pass needs)."""
    norm = F.f8f8bf16_rmsnorm_quantize(x, w.norm, residual=residual, want_y=True, want_rstd=True)
    logits = norm.Y.float() @ w.router.t()
    route = F.f8f8bf16_route(logits, k, bias=w.bias, score="sigmoid")
    rows, scales = F.f8f8bf16_moe_dispatch(norm.XQ, norm.x_scale, route.dst_row)
    h = F.f8f8bf16_rowwise_grouped_stacked(rows, q["w1"][0], scales, q["w1"][1], route.M_sizes)
    act = F.f8f8bf16_silu_mul_quantize(h, checkpoint=True)
    y = F.f8f8bf16_rowwise_grouped_stacked(act.AQ, q["w2"][0], act.a_scale, q["w2"][1], route.M_sizes)
    out = F.f8f8bf16_moe_combine(y, route.dst_row, route.weights)
    return out, norm.residual, (norm, logits, route, rows, scales, act, y)


def backward(dout, dresidual, w: Weights, q: dict, kept):
    """Gradients of (input and residual, norm weight, router weight, w1, w2)."""
    norm, logits, route, rows, scales, act, y = kept
    M = route.M_sizes
    dy, dweights = F.f8f8bf16_moe_combine_backward(dout, route.dst_row, route.weights, y)
    # down product: its input's gradient, and dW2 = dY^T A per expert
    dyq, dys = F.f8f8bf16_quantize_rowwise(dy)
    da = F.f8f8bf16_rowwise_grouped_stacked(dyq, q["w2t"][0], dys, q["w2t"][1], M)
    dyt, dyt_s, ko = F.f8f8bf16_quantize_k_offsets(dy, M)
    at, at_s, _ = F.f8f8bf16_quantize_k_offsets(act.AQ, M, x_scale=act.a_scale)
    dw2 = F.f8f8bf16_rowwise_grouped_k_offsets(dyt, at, dyt_s, at_s, ko)
    # gated activation, from its 8-bit checkpoint
    dh = F.f8f8bf16_silu_mul_backward(da, act.HQ, act.h_scale)
    # gate and up product: its input's gradient, and dW1 = dH^T X per expert
    dhq, dhs = F.f8f8bf16_quantize_rowwise(dh)
    drows = F.f8f8bf16_rowwise_grouped_stacked(dhq, q["w1t"][0], dhs, q["w1t"][1], M)
    dht, dht_s, ko = F.f8f8bf16_quantize_k_offsets(dh, M)
    xt, xt_s, _ = F.f8f8bf16_quantize_k_offsets(rows, M, x_scale=scales)
    dw1 = F.f8f8bf16_rowwise_grouped_k_offsets(dht, xt, dht_s, xt_s, ko)
    # the router, and both gradients of the normalised rows together
    dlogits = F.f8f8bf16_route_backward(logits, route.ids, dweights, score="sigmoid")
    drouter = dlogits.t() @ norm.Y.float()
    dnorm = F.f8f8bf16_moe_combine(drows, route.dst_row, addend=(dlogits @ w.router).to(torch.bfloat16))
    dx, dnorm_w = F.f8f8bf16_rmsnorm_backward(dnorm, norm.residual, w.norm, norm.rstd, dresidual=dresidual)
    return dx, dnorm_w, drouter, dw1, dw2


def train_operands(w: Weights, fp8: bool) -> dict:
    """The products' operands of one step, from the fp32 weights: codes with a scale per 128 x 128
    values, as they are and transposed, or bf16, whose products read one layout in both passes."""
    if fp8:
        return {n: F.f8f8bf16_quantize_groupwise_weight(getattr(w, n), transposed=True) for n in ("w1", "w2")}
    return {n: getattr(w, n).to(torch.bfloat16) for n in ("w1", "w2")}


def train_product(rows, rows_bf16, q, M_sizes):
    """rows (codes and scales, which fp8 products read) or the same in bf16, times an expert weight."""
    if isinstance(q, F.WeightBlocks):
        return F.f8f8bf16_groupwise_grouped_stacked(rows[0], q.WQ, rows[1], q.w_scale, M_sizes)
    return F.bf16_grouped_stacked(rows_bf16, q, M_sizes)


def train_dgrad(dy, q, M_sizes):
    """The gradient of train_product's rows."""
    if isinstance(q, F.WeightBlocks):
        dyq, dys = F.f8f8bf16_quantize_groupwise(dy)
        return F.f8f8bf16_groupwise_grouped_stacked(dyq, q.WQt, dys, q.wt_scale, M_sizes)
    return F.bf16_grouped_stacked_dgrad(dy, q, M_sizes)


def gated(h):
    """silu(gate) * up of bf16 rows [gate | up], in fp32, rounded once."""
    gate, up = h.float().chunk(2, 1)
    return (torch.nn.functional.silu(gate) * up).to(torch.bfloat16)


def gated_backward(da, h):
    """Its gradient from the rows themselves."""
    gate, up = h.float().chunk(2, 1)
    sig, d = torch.sigmoid(gate), da.float()
    return torch.cat([d * up * sig * (1 + gate * (1 - sig)), d * gate * sig], 1).to(torch.bfloat16)


def train_forward(x, residual, w: Weights, q: dict, k: int):
    """forward with the operands of train_operands: hidden and inner sizes that are multiples of 128."""
    norm = F.f8f8bf16_rmsnorm_quantize(x, w.norm, residual=residual, block=128, want_y=True, want_rstd=True)
    logits = norm.Y.float() @ w.router.t()
    route = F.f8f8bf16_route(logits, k, bias=w.bias, score="sigmoid")
    rows = F.f8f8bf16_moe_dispatch(norm.XQ, norm.x_scale, route.dst_row)
    xb, _ = F.f8f8bf16_moe_combine_backward(norm.Y, route.dst_row)       # the same rows in bf16
    h = train_product(rows, xb, q["w1"], route.M_sizes)
    if isinstance(q["w2"], F.WeightBlocks):
        act = F.f8f8bf16_silu_mul_quantize(h, block=128, checkpoint=True)
        ab = (act.AQ.view(torch.float8_e4m3fn).float().unflatten(1, (-1, 128)) * act.a_scale[:, :, None]).flatten(1).to(torch.bfloat16)
    else:
        act, ab = h, gated(h)
    y = train_product(act, ab, q["w2"], route.M_sizes)
    out = F.f8f8bf16_moe_combine(y, route.dst_row, route.weights)
    return out, norm.residual, (norm, logits, route, xb, act, ab, y)


def train_backward(dout, dresidual, w: Weights, q: dict, kept, grads: dict):
    """Adds the weights' gradients to `grads` (fp32) and returns that of input and residual."""
    norm, logits, route, xb, act, ab, y = kept
    M = route.M_sizes
    dy, dweights = F.f8f8bf16_moe_combine_backward(dout, route.dst_row, route.weights, y)
    da = train_dgrad(dy, q["w2"], M)
    F.bf16_grouped_stacked_wgrad(dy, ab, M, dW=grads["w2"], accumulate=True)
    dh = gated_backward(da, act) if torch.is_tensor(act) else F.f8f8bf16_silu_mul_backward(da, act.HQ, act.h_scale)
    drows = train_dgrad(dh, q["w1"], M)
    F.bf16_grouped_stacked_wgrad(dh, xb, M, dW=grads["w1"], accumulate=True)
    dlogits = F.f8f8bf16_route_backward(logits, route.ids, dweights, score="sigmoid")
    grads["router"] += dlogits.t() @ norm.Y.float()
    dnorm = F.f8f8bf16_moe_combine(drows, route.dst_row, addend=(dlogits @ w.router).to(torch.bfloat16))
    dx, dnorm_w = F.f8f8bf16_rmsnorm_backward(dnorm, norm.residual, w.norm, norm.rstd, dresidual=dresidual)
    grads["norm"] += dnorm_w
    return dx


def train_step(batches, w: Weights, k: int, lr: float = 1e-3, max_norm: float = 1.0, fp8: bool = True):
    """One step of plain gradient descent over micro-batches, each (x, residual, gradients of the layer's two
    outputs), with the gradients clipped by their common norm.  Returns (the clipped gradients, norm)."""
    q = train_operands(w, fp8)
    grads = {n: torch.zeros_like(getattr(w, n)) for n in ("norm", "router", "w1", "w2")}
    for x, residual, dout, dresidual in batches:
        _, _, kept = train_forward(x, residual, w, q, k)
        train_backward(dout, dresidual, w, q, kept, grads)
    norm = F.f8f8bf16_grad_clip(list(grads.values()), max_norm)
    for n, g in grads.items():
        getattr(w, n).sub_(g, alpha=lr)
    return grads, norm


def reference(x, residual, w: Weights, ids, dout, dresidual):
    """The same layer in fp32, the choice of experts given: (output, gradients)."""
    h = (x.float() + residual.float()).to(torch.bfloat16).float().requires_grad_(True)
    p = [t.clone().requires_grad_(True) for t in (w.norm, w.router, w.w1, w.w2)]
    norm, router, w1, w2 = p
    y = h * torch.rsqrt((h * h).mean(1, keepdim=True) + 1e-6) * norm
    score = torch.sigmoid(y @ router.t()).gather(1, ids)
    weights = score / score.sum(1, keepdim=True)
    out = torch.zeros_like(h)
    for e in range(w1.shape[0]):
        t, j = (ids == e).nonzero(as_tuple=True)
        if t.numel():
            gate, up = (y[t] @ w1[e].t()).chunk(2, dim=1)
            out = out.index_add(0, t, ((torch.nn.functional.silu(gate) * up) @ w2[e].t()) * weights[t, j, None])
    grads = torch.autograd.grad([out, h], [h, norm, router, w1, w2], [dout.float(), dresidual.float()])
    return out.detach(), grads


def main() -> None:
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--tokens", type=int, default=512)
    ap.add_argument("--hidden", type=int, default=1024)
    ap.add_argument("--inner", type=int, default=512)
    ap.add_argument("--experts", type=int, default=16)
    ap.add_argument("--topk", type=int, default=4)
    ap.add_argument("--steps", type=int, default=20)
    a = ap.parse_args()
    w = random_weights(a.hidden, a.inner, a.experts)
    q = w.quantized()
    g = torch.Generator(device="cuda").manual_seed(1)
    x, residual, dout, dres = (torch.randn(a.tokens, a.hidden, generator=g, device="cuda").to(torch.bfloat16) for _ in range(4))
    out, _, kept = forward(x, residual, w, q, a.topk)
    grads = backward(dout, dres, w, q, kept)
    want, want_grads = reference(x, residual, w, kept[2].ids.long(), dout, dres)
    for name, got, ref in zip(("output", "input", "norm weight", "router", "w1", "w2"), (out, *grads), (want, *want_grads)):
        print(f"{name:12s} relative difference to fp32: {float((got.float() - ref).norm() / ref.norm()):.4f}")

    def timed(f):
        for _ in range(3):
            f()
        torch.cuda.synchronize()
        t = time.perf_counter()
        for _ in range(a.steps):
            f()
        torch.cuda.synchronize()
        return (time.perf_counter() - t) / a.steps * 1e6
    print(f"forward  {timed(lambda: forward(x, residual, w, q, a.topk)):9.1f} us")
    print(f"backward {timed(lambda: backward(dout, dres, w, q, kept)):9.1f} us")
    if a.hidden % 128 == 0 and a.inner % 128 == 0:
        batch = [(x, residual, dout, dres)]
        for fp8 in (True, False):
            us = timed(lambda: train_step(batch, w, a.topk, fp8=fp8))
            print(f"training step, {'fp8' if fp8 else 'bf16'} products {us:9.1f} us")


if __name__ == "__main__":
    main()
