"""CPU-only checks of the layer operators' C ABI and binding: exports, sizes of
workspaces, and refusals before anything reaches the GPU (the addresses are never
dereferenced)."""
import os
import re

import pytest
import torch

import fp8_rowwise_scaled_amd as F
from fp8_rowwise_scaled_amd import _lib

HEADER = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include", "fp8gg_layer.h")
M = 1 << 24
A = [0x10000000 + i * M for i in range(12)]     # twelve far-apart fake addresses
BAD, SHAPE, OK = _lib.ERR_INVALID_ARGUMENT, _lib.ERR_UNSUPPORTED_SHAPE, _lib.OK


def lib():
    return _lib.load()


def test_library_exports_every_declared_symbol():
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    names = set(re.findall(r"\b(f8f8bf16_\w+)\s*\(", text))
    assert names == set(_lib.LAYER_EXPORTS)
    for n in names:
        assert hasattr(lib(), n), n


def norm(X=A[0], res=None, w=A[1], wt=0, eps=1e-6, block=0, q=A[2], s=A[3], y=None, ro=None, rstd=None, rows=4, K=128):
    return lib().f8f8bf16_rmsnorm_quantize(X, res, w, wt, eps, block, q, s, y, ro, rstd, rows, K, None)


@pytest.mark.parametrize("kw,status,text", [
    (dict(K=12), SHAPE, "multiple of 8"), (dict(K=0), SHAPE, "positive"), (dict(K=32776), SHAPE, "exceeds"),
    (dict(rows=-1), BAD, "negative"), (dict(block=64), BAD, "block=64"), (dict(block=128, K=136), SHAPE, "multiple of 128"),
    (dict(wt=2), BAD, "weight_dtype"), (dict(eps=-1.0), BAD, "eps"), (dict(eps=float("nan")), BAD, "eps"),
    (dict(eps=float("inf")), BAD, "eps"), (dict(res=A[4]), BAD, "together"), (dict(ro=A[4]), BAD, "together"),
    (dict(X=None), BAD, "X is null"), (dict(X=A[0] + 8), BAD, "16-byte"), (dict(q=A[2] + 4), BAD, "8-byte"),
    (dict(s=A[0] + 64), BAD, "overlaps"), (dict(res=A[4], ro=A[4] + 16), BAD, "overlaps"),
    (dict(res=A[4], ro=A[0]), BAD, "overlaps"), (dict(y=A[0]), BAD, "overlaps"), (dict(rows=1 << 45), SHAPE, "too large"),
    (dict(rows=0, X=None, w=None, q=None, s=None), OK, ""),
])
def test_norm_refusals(kw, status, text):
    assert norm(**kw) == status and text in F.layer_last_error()


def test_norm_backward_refusals():
    def call(dy=A[0], h=A[1], w=A[2], wt=0, r=A[3], dres=None, dx=A[4], dw=A[5], ws=A[6], size=1 << 20, rows=4, K=128):
        return lib().f8f8bf16_rmsnorm_backward(dy, h, w, wt, r, dres, dx, dw, ws, size, rows, K, None)
    need = lib().f8f8bf16_rmsnorm_backward_workspace(4, 128)
    assert need > 0 and lib().f8f8bf16_rmsnorm_backward_workspace(0, 128) == 0
    assert call(size=need - 1) == BAD and "workspace" in F.layer_last_error()
    assert call(ws=None) == BAD and "workspace" in F.layer_last_error()
    assert call(dx=A[1]) == BAD and "overlaps" in F.layer_last_error()       # dX may be dY, not H
    assert call(dw=A[5] + 4) == BAD and call(K=4) == SHAPE and call(wt=7) == BAD and call(rows=-2) == BAD


def route(x=A[0], dt=1, b=None, score=0, ng=1, tg=1, gt=1, w=A[1], i=A[2], m=A[3], d=A[4], ws=A[5], size=1 << 22, T=64,
          E=32, k=4, scale=1.0):
    return lib().f8f8bf16_route(x, dt, b, score, ng, tg, gt, 1, scale, w, i, m, d, ws, size, T, E, k, None)


@pytest.mark.parametrize("kw,status,text", [
    (dict(dt=2), BAD, "logits_dtype"), (dict(score=2), BAD, "score"), (dict(E=0, k=0), SHAPE, "E=0"),
    (dict(E=1025), SHAPE, "E=1025"), (dict(k=0), SHAPE, "k=0"), (dict(k=17), SHAPE, "k=17"), (dict(E=3), SHAPE, "k=4"),
    (dict(ng=5), SHAPE, "n_group"), (dict(ng=0), SHAPE, "n_group"), (dict(ng=32), SHAPE, "n_group"),
    (dict(ng=4, tg=5), BAD, "topk_group"), (dict(tg=0), BAD, "topk_group"), (dict(gt=3), BAD, "group_top"),
    (dict(scale=float("nan")), BAD, "scale"), (dict(m=None), BAD, "together"), (dict(d=None), BAD, "together"),
    (dict(T=1 << 31), SHAPE, "too large"),
    (dict(T=4096, size=0), BAD, "workspace"), (dict(T=4096, ws=None), BAD, "workspace"),
    (dict(x=A[0] + 4), BAD, "16-byte"), (dict(w=A[0]), BAD, "overlaps"), (dict(T=-1), BAD, "negative"),
    (dict(T=0, m=None, d=None, x=None, w=None, i=None), OK, ""),
])
def test_route_refusals(kw, status, text):
    assert route(**kw) == status and text in F.layer_last_error()


def test_route_workspace():
    """Counts of at most 256 workgroups, however many tokens; none for a few pairs."""
    ws = lib().f8f8bf16_route_workspace
    assert ws(64, 256, 8) == 0 and ws(512, 256, 8) == 0 and ws(513, 256, 8) >= 2 * 256 * 4 and ws(5000, 9, 1) >= 2 * 9 * 4
    assert ws(16384, 256, 8) == ws(1 << 20, 256, 8) == 256 * 256 * 4


def test_route_backward_refusals():
    def call(x=A[0], dt=1, i=A[1], dw=A[2], dx=A[3], T=4, E=32, k=4):
        return lib().f8f8bf16_route_backward(x, dt, i, dw, 0, 1, 1.0, dx, T, E, k, None)
    assert call(dt=5) == BAD and call(k=33) == SHAPE and call(dx=A[0]) == BAD and call(i=None) == BAD
    assert call(T=0, x=None, i=None, dw=None, dx=None) == OK


def test_exchange_refusals():
    def dispatch(q=A[0], s=A[1], cols=1, d=A[2], o=A[3], so=A[4], T=4, k=2, R=8, K=128):
        return lib().f8f8bf16_moe_dispatch(q, s, cols, d, o, so, T, k, R, K, None)
    assert dispatch(K=120) == SHAPE and dispatch(k=65) == SHAPE and dispatch(cols=0) == BAD and dispatch(R=-1) == BAD
    assert dispatch(o=A[0]) == BAD and dispatch(d=None) == BAD and dispatch(so=A[3]) == BAD and dispatch(q=A[0] + 8) == BAD
    assert dispatch(T=0, q=None, s=None, d=None, o=None, so=None) == OK

    def combine(y=A[0], d=A[1], w=A[2], add=None, o=A[3], T=4, k=2, R=8, N=128):
        return lib().f8f8bf16_moe_combine(y, d, w, add, o, T, k, R, N, None)
    assert combine(N=12) == SHAPE and combine(N=0) == SHAPE and combine(o=A[0]) == BAD and combine(o=None) == BAD
    assert combine(add=A[4], o=A[4] + 16) == BAD and combine(T=1 << 31) == SHAPE and combine(T=0, y=None, o=None) == OK

    def back(do=A[0], d=A[1], w=A[2], y=A[3], dy=A[4], dw=A[5], T=4, k=2, R=8, N=128):
        return lib().f8f8bf16_moe_combine_backward(do, d, w, y, dy, dw, T, k, R, N, None)
    assert back(dw=None) == BAD and back(y=None) == BAD and "together" in F.layer_last_error()
    assert back(dy=A[0]) == BAD and back(dy=A[3] + 256) == BAD and back(N=4) == SHAPE and back(k=0) == OK


def test_checkpoint_refusals():
    def fwd(h=A[0], block=0, q=A[1], s=A[2], hq=None, hs=None, rows=4, I=128):
        return lib().f8f8bf16_silu_mul_quantize(h, block, q, s, hq, hs, rows, I, None)
    assert fwd(I=12) == SHAPE and fwd(block=128, I=136) == SHAPE and fwd(block=1) == BAD and fwd(hq=A[3]) == BAD
    assert fwd(q=A[0]) == BAD and fwd(I=40000) == SHAPE and fwd(s=None) == BAD and fwd(rows=0, h=None, q=None, s=None) == OK

    def back(da=A[0], hq=A[1], hs=A[2], dh=A[3], rows=4, I=128):
        return lib().f8f8bf16_silu_mul_backward(da, hq, hs, dh, rows, I, None)
    assert back(dh=A[0]) == BAD and back(hs=None) == BAD and back(I=4) == SHAPE and back(rows=-1) == BAD

    def ko(x=A[0], dt=2, s=A[1], cols=1, m=A[2], xt=A[3], ts=A[4], o=A[5], ws=A[6], size=1 << 20, R=64, G=4, K=256):
        return lib().f8f8bf16_quantize_k_offsets(x, dt, s, cols, m, xt, ts, o, ws, size, R, G, K, None)
    assert ko(dt=1) == BAD and ko(s=None) == BAD and ko(cols=3) == BAD and ko(dt=0) == BAD and "none" in F.layer_last_error()
    assert ko(K=24) == SHAPE and ko(G=0) == SHAPE and ko(G=1025) == SHAPE and ko(size=16) == BAD and ko(xt=A[0]) == BAD
    assert ko(m=None) == BAD and ko(xt=A[3] + 8) == BAD and ko(R=(1 << 31) - 300, size=1 << 50) == SHAPE


def test_k_offsets_capacity_holds_every_split():
    cap = F.f8f8bf16_k_offsets_capacity
    assert cap(0, 4) == 0 and cap(1, 4) == 16 and cap(3, 8) == 48 and cap(64, 1) == 80 and cap(4096, 8) == 4224
    for R in range(1, 40):                       # the worst split: as many groups of 16 n + 1 rows as there are
        for G in range(1, 6):
            worst = 16 * (min(R, G) - 1) + -(-(R - min(R, G) + 1) // 16) * 16
            assert worst <= cap(R, G) and cap(R, G) % 16 == 0


def test_binding_refuses_before_the_library():
    x = torch.zeros((4, 128), dtype=torch.bfloat16)
    w = torch.zeros(128)
    with pytest.raises(ValueError, match="on the GPU"):
        F.f8f8bf16_rmsnorm_quantize(x, w)
    with pytest.raises(ValueError, match="bfloat16"):
        F.f8f8bf16_rmsnorm_quantize(x.float(), w)
    with pytest.raises(ValueError, match=r"\[rows, K\]"):
        F.f8f8bf16_rmsnorm_quantize(x[0], w)
    with pytest.raises(ValueError, match="bfloat16 or float32"):
        F.f8f8bf16_route(x.double(), 2)
    with pytest.raises(ValueError, match="on the GPU"):
        F.f8f8bf16_route(x, 2)
    with pytest.raises(ValueError):
        F.f8f8bf16_moe_combine(x, torch.zeros((4,), dtype=torch.int32))


def test_layer_error_is_per_thread_and_cleared():
    import threading
    assert norm(K=12) == SHAPE and F.layer_last_error()
    seen = []
    t = threading.Thread(target=lambda: seen.append(F.layer_last_error()))
    t.start()
    t.join()
    assert seen == [""]
    assert norm(rows=0) == OK and F.layer_last_error() == ""


def test_missing_binding_raises(monkeypatch):
    """There is no fallback: without the compiled module the calls raise."""
    from fp8_rowwise_scaled_amd import layer

    def gone(name, package=None):
        raise ImportError("no such file")
    monkeypatch.setattr(layer, "_module", None)
    monkeypatch.setattr(layer.importlib, "import_module", gone)
    with pytest.raises(RuntimeError, match="no fallback"):
        F.f8f8bf16_moe_combine(torch.zeros((4, 16), dtype=torch.bfloat16), torch.zeros((2, 2), dtype=torch.int32))


def test_arguments_of_the_wrong_kind():
    with pytest.raises(ValueError, match="must be a tensor"):
        F.f8f8bf16_moe_combine([1, 2], None)
    with pytest.raises(ValueError, match="must be a tensor"):
        F.f8f8bf16_route(None, 2)

