"""CPU-only checks of the training operators' C ABI and binding: exports, sizes of
workspaces, and refusals before anything reaches the GPU (the addresses are never
dereferenced)."""
import ctypes
import os
import re
import subprocess
import sys

import pytest
import torch

import fp8_rowwise_scaled_amd as F
from fp8_rowwise_scaled_amd import _lib

HEADER = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include", "fp8gg_train.h")
M = 1 << 24
A = [0x10000000 + i * M for i in range(12)]     # twelve far-apart fake addresses
BAD, SHAPE, OK = _lib.ERR_INVALID_ARGUMENT, _lib.ERR_UNSUPPORTED_SHAPE, _lib.OK


def lib():
    return _lib.load()


def test_library_exports_every_declared_symbol():
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    names = set(re.findall(r"\b(f8f8bf16_\w+|bf16_\w+)\s*\(", text))
    assert names == set(_lib.TRAIN_EXPORTS)
    for n in names:
        assert hasattr(lib(), n), n


PRODUCT = [
    (dict(N=12), SHAPE, "multiples of 8"), (dict(K=4), SHAPE, "multiples of 8"), (dict(G=-1), BAD, "negative"),
    (dict(M=-1), BAD, "negative"), (dict(M=1 << 31), SHAPE, "too large"), (dict(N=1 << 23), SHAPE, "too large"),
    (dict(K=1 << 23), SHAPE, "too large"), (dict(G=1 << 20, N=1 << 22, K=1 << 22), SHAPE, "2^47"),
    (dict(p=None), BAD, "is null"), (dict(w=None), BAD, "W is null"), (dict(m=None), BAD, "M_sizes is null"),
    (dict(o=None), BAD, "is null"), (dict(p=A[0] + 8), BAD, "16-byte"), (dict(w=A[1] + 2), BAD, "16-byte"),
    (dict(m=A[2] + 4), BAD, "8-byte"), (dict(o=A[3] + 4), BAD, "16-byte"), (dict(o=A[0]), BAD, "overlaps"),
    (dict(o=A[1] + 16), BAD, "overlaps W"), (dict(o=A[2]), BAD, "overlaps M_sizes"),
    (dict(M=0, p=None, o=None), OK, ""), (dict(G=0, w=None, m=None), OK, ""),
]


@pytest.mark.parametrize("name", ["bf16_grouped_stacked", "bf16_grouped_stacked_dgrad"])
@pytest.mark.parametrize("kw,status,text", PRODUCT)
def test_product_refusals(name, kw, status, text):
    def call(p=A[0], w=A[1], m=A[2], o=A[3], G=4, M=64, N=128, K=256):
        return getattr(lib(), name)(p, w, m, o, G, M, N, K, None)
    assert call(**kw) == status and text in F.layer_last_error()


def test_product_refuses_more_tiles_than_a_launch_holds():
    big = 1 << 60
    assert lib().bf16_grouped_stacked(big, 2 * big, A[2], 3 * big, 1 << 24, (1 << 31) - 65536, 1 << 14, 8, None) == SHAPE
    assert "workgroups" in F.layer_last_error()


def test_wgrad_refusals():
    def call(dy=A[0], x=A[1], m=A[2], dw=A[3], dt=1, acc=0, ws=None, size=0, G=8, M=64, N=128, K=256):
        return lib().bf16_grouped_stacked_wgrad(dy, x, m, dw, dt, acc, ws, size, G, M, N, K, None)
    assert call(dt=2) == BAD and "dw_dtype" in F.layer_last_error()
    assert call(dt=0, acc=1) == BAD and "accumulate" in F.layer_last_error()
    assert call(dw=A[0]) == BAD and call(dw=A[1]) == BAD and call(dw=None) == BAD and call(x=A[1] + 8) == BAD
    assert call(N=4) == SHAPE and call(K=-8) == BAD and call(m=None) == BAD
    assert call(G=0, m=None, dw=None) == OK
    need = lib().bf16_grouped_stacked_wgrad_workspace(1, 8192, 128, 256)
    assert need > 0 and need % (128 * 256 * 4) == 0
    assert call(G=1, M=8192) == BAD and "workspace" in F.layer_last_error()
    assert call(G=1, M=8192, ws=A[4], size=need - 1) == BAD
    assert call(G=1, M=8192, ws=A[4] + 8, size=need) == BAD and "16-byte" in F.layer_last_error()
    assert call(G=1, M=8192, ws=A[3], size=need) == BAD and "overlaps" in F.layer_last_error()


def test_fp32_weight_gradients_past_the_largest_tensor():
    """2^47 bytes are 2^45 fp32 values."""
    def call(dt, G):
        return lib().bf16_grouped_stacked_wgrad(A[0], A[1], A[2], A[0], dt, 0, None, 0, G, 8, 1 << 22, 1 << 20, None)
    assert call(1, 9) == SHAPE and "2^47" in F.layer_last_error()
    assert call(1, 8) == BAD and "overlaps" in F.layer_last_error()          # passes the sizes' check
    assert call(0, 16) == BAD and "overlaps" in F.layer_last_error()
    assert call(0, 17) == SHAPE and "2^47" in F.layer_last_error()


def test_wgrad_workspace():
    """Sums of parts only where a few tiles meet many rows, and never more than 32 of them."""
    ws = lib().bf16_grouped_stacked_wgrad_workspace
    assert ws(8, 4096, 4096, 7168) == 0 and ws(1, 64, 128, 128) == 0 and ws(0, 64, 128, 128) == 0 and ws(1, 0, 128, 128) == 0
    assert ws(1, 1 << 20, 128, 128) == 32 * 128 * 128 * 4 and ws(-1, 5, 8, 8) == 0
    assert ws(1, 1024, 256, 128) == 4 * 256 * 128 * 4


@pytest.mark.parametrize("sizes", [(1 << 32, 1 << 40, 1 << 40, 8), (1, 1 << 20, (1 << 63) - 1, 8), ((1 << 63) - 1,) * 4, (1, -(1 << 63), 8, 8),
                                   (1 << 31, 1 << 30, 8, 8), (1, 1 << 31, 8, 8), (1, 4096, 1 << 23, 8), (1, 4096, 8, 1 << 23)])
def test_wgrad_workspace_of_sizes_that_are_refused(sizes):
    """0, in a process of its own: products of such sizes have wrapped to 0 and been divided by."""
    code = f"from fp8_rowwise_scaled_amd import _lib; print(_lib.load().bf16_grouped_stacked_wgrad_workspace(*{sizes}))"
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, cwd=os.path.dirname(os.path.dirname(HEADER)), timeout=120)
    assert (r.returncode, r.stdout.strip()) == (0, "0"), r.stderr


def test_quantize_refusals():
    def rows(x=A[0], q=A[1], s=A[2], rows=4, K=256):
        return lib().f8f8bf16_quantize_groupwise(x, q, s, rows, K, None)
    assert rows(K=0) == SHAPE and rows(K=192) == SHAPE and rows(rows=-1) == BAD and rows(q=A[0]) == BAD
    assert rows(x=A[0] + 8) == BAD and rows(q=A[1] + 8) == BAD and rows(s=A[2] + 2) == BAD and rows(s=None) == BAD
    assert rows(rows=1 << 45) == SHAPE and rows(rows=0, x=None, q=None, s=None) == OK

    def weight(w=A[0], dt=1, q=A[1], s=A[2], qt=A[3], st=A[4], G=2, N=128, K=256):
        return lib().f8f8bf16_quantize_groupwise_weight(w, dt, q, s, qt, st, G, N, K, None)
    assert weight(dt=2) == BAD and weight(N=64) == SHAPE and weight(K=130) == SHAPE and weight(G=-1) == BAD
    assert weight(qt=None) == BAD and weight(st=None) == BAD and "together" in F.layer_last_error()
    assert weight(q=A[0]) == BAD and weight(qt=A[1] + 128) == BAD and weight(st=A[2]) == BAD and weight(w=None) == BAD
    assert weight(qt=A[3] + 8) == BAD and weight(G=1 << 24, N=1 << 14, K=1 << 14) == SHAPE
    assert weight(G=0, w=None, q=None, s=None, qt=None, st=None) == OK


def test_weight_blocks_refused_past_a_launch():
    """A workgroup of 256 threads per block, and fewer than 2^32 threads in a launch."""
    big = 1 << 50
    def weight(N, K, G=1, t=True):
        return lib().f8f8bf16_quantize_groupwise_weight(big, 0, 2 * big, A[0], 3 * big if t else None, A[1] if t else None, G, N, K, None)
    for G, N, K in ((1, 128 << 12, 128 << 12), (1 << 24, 128, 128), (3, 128 << 12, 128 << 11)):
        for t in (True, False):
            assert weight(N, K, G, t) == SHAPE and "too large" in F.layer_last_error()
    # one block fewer passes the checks (and meets the addresses' overlap)
    assert weight(128, 128, (1 << 24) - 1) == BAD and "overlaps" in F.layer_last_error()


def table(*tensors):
    """(grads, counts, dtypes, n) of (address, count, dtype) triples."""
    n = len(tensors)
    return ((ctypes.c_void_p * n)(*[t[0] for t in tensors]), (ctypes.c_int64 * n)(*[t[1] for t in tensors]),
            (ctypes.c_int32 * n)(*[t[2] for t in tensors]), n)


def test_square_sum_refusals():
    def call(*tensors, out=A[8], ws=A[9], size=1 << 20):
        g, c, d, n = table(*tensors)
        return lib().f8f8bf16_grad_square_sum(g, c, d, n, out, ws, size, None)
    ok = (A[0], 100, 1)
    assert call((A[0], 100, 2)) == BAD and "dtypes[0]" in F.layer_last_error()
    assert call(ok, (A[1], -1, 0)) == BAD and "counts[1]" in F.layer_last_error()
    assert call(ok, (None, 4, 0)) == BAD and "grads[1]" in F.layer_last_error()
    assert call((A[0] + 2, 100, 1)) == BAD and "aligned" in F.layer_last_error()
    assert call(ok, out=None) == BAD and call(ok, out=A[8] + 4) == BAD and call(ok, ws=None) == BAD
    assert call(ok, size=lib().f8f8bf16_grad_workspace(1) - 1) == BAD and "workspace" in F.layer_last_error()
    assert call(ok, out=A[0] + 80) == BAD and "square_sum overlaps grads[0]" in F.layer_last_error()
    assert call(ok, out=A[9]) == BAD and call((A[9] + 64, 4, 0)) == BAD
    assert lib().f8f8bf16_grad_square_sum(None, None, None, -1, A[8], A[9], 1 << 20, None) == BAD
    assert lib().f8f8bf16_grad_square_sum(None, None, None, 1, A[8], A[9], 1 << 20, None) == BAD


@pytest.mark.parametrize("dtype,most", [(1, (0x7FFFFFFF // 96) * 4096), (0, (0x7FFFFFFF // 96) * 8192)])
def test_gradients_past_a_launch(dtype, most):
    """96 tensors' chunks of 16 KB are counted in 32 bits: tensors of more than 366 GB are refused (they wrapped the count)."""
    def call(count):
        g, c, d, n = table((A[0], count, dtype))
        return lib().f8f8bf16_grad_square_sum(g, c, d, n, A[0], A[9], 1 << 20, None)
    assert call(most) == BAD and "square_sum overlaps grads[0]" in F.layer_last_error()     # passes the sizes' check
    for count in (most + 1, 1 << 43, (1 << 44) - 1, 1 << 44, (1 << 63) - 1):
        assert call(count) == SHAPE and "counts[0]" in F.layer_last_error(), count


def test_clip_refusals():
    def call(*tensors, outs=None, sum_=None, bound=1.0, eps=0.0, norm=A[8], ws=A[9], size=1 << 20):
        g, c, d, n = table(*tensors)
        o = (ctypes.c_void_p * n)(*(outs or [t[0] for t in tensors]))
        return lib().f8f8bf16_grad_clip(g, o, c, d, n, sum_, bound, eps, norm, ws, size, None)
    a, b = (A[0], 100, 1), (A[1], 100, 0)
    nan = float("nan")
    assert call(a, bound=-1.0) == BAD and call(a, bound=nan) == BAD and call(a, eps=-1.0) == BAD and call(a, eps=nan) == BAD
    assert call(a, eps=float("inf")) == BAD and call(a, norm=None) == BAD and call(a, norm=A[8] + 2) == BAD
    assert call(a, norm=A[0]) == BAD and "norm overlaps grads[0]" in F.layer_last_error()
    assert call(a, outs=[A[2]], norm=A[2] + 4) == BAD and "norm overlaps outs[0]" in F.layer_last_error()
    assert call(a, sum_=A[0]) == BAD and call(a, size=8) == BAD and call(a, sum_=A[7] + 4) == BAD
    # the same tensor twice, or outputs that meet another tensor
    assert call(a, a) == BAD and "outs[" in F.layer_last_error()
    assert call(a, b, outs=[A[2], A[2] + 396]) == BAD and call(a, b, outs=[A[1], A[2]]) == BAD
    assert call(a, b, outs=[A[2], A[0] + 396]) == BAD and "grads[0]" in F.layer_last_error()
    assert call(a, outs=[A[0] + 4]) == BAD and call(a, outs=[A[2] + 2]) == BAD and "aligned" in F.layer_last_error()
    assert call((A[0], 1000, 1), (A[0] + 8, 2, 1), outs=[A[2], A[0] + 3996]) == BAD


def test_grad_workspace():
    ws = lib().f8f8bf16_grad_workspace
    assert ws(0) == 0 and ws(-3) == 0 and ws(1) == ws(96) and ws(97) == 2 * (ws(1) - 8) + 8 and ws(1) % 8 == 0


def test_binding_refuses_before_the_library():
    x = torch.zeros((4, 128), dtype=torch.bfloat16)
    w = torch.zeros((2, 64, 128), dtype=torch.bfloat16)
    m = torch.zeros(2, dtype=torch.int64)
    for call, text in [
            (lambda: F.bf16_grouped_stacked(x, w, m), "on the GPU"),
            (lambda: F.bf16_grouped_stacked(x.float(), w, m), "bfloat16"),
            (lambda: F.bf16_grouped_stacked(x[0], w, m), r"\[total_M, K\]"),
            (lambda: F.bf16_grouped_stacked(None, w, m), "must be a tensor"),
            (lambda: F.bf16_grouped_stacked_dgrad(x, w, None), "must be a tensor"),
            (lambda: F.bf16_grouped_stacked_wgrad(x, x, m, dtype=torch.float16), "dtype"),
            (lambda: F.bf16_grouped_stacked_wgrad(x, x, m), "on the GPU"),
            (lambda: F.f8f8bf16_quantize_groupwise(x.float()), "bfloat16"),
            (lambda: F.f8f8bf16_quantize_groupwise_weight(w.half()), "bfloat16 or float32"),
            (lambda: F.f8f8bf16_grad_square_sum(x), "list or tuple"),
            (lambda: F.f8f8bf16_grad_square_sum(None), "list or tuple"),
            (lambda: F.f8f8bf16_grad_clip([x, None], 1.0), r"grads\[1\] must be a tensor"),
            (lambda: F.f8f8bf16_grad_clip([x.half()], 1.0), "bfloat16 or float32"),
            (lambda: F.f8f8bf16_grad_clip([x], 1.0), "on the GPU")]:
        with pytest.raises(ValueError, match=text):
            call()
