"""Refusals of the operators with 128-element scales, on a host without a GPU:
every call fails validation (or is empty) before any CUDA call."""

import pytest
import torch

OK, INVALID, SHAPE, ALIGN, UNSUPPORTED = 0, 1, 2, 3, 4
A = 0x10000          # an aligned fake device address (never dereferenced)
E4M3, E5M2 = 1, 2
BLOCK, POW2 = 1 << 10, 1 << 11
BF16, FP16, FP32 = 0, 1, 2


def quant(mx, **kw):
    a = dict(x=A, dtype=BF16, rows=4, cols=256, ldx=256, format=E4M3, flags=0, codes=A, ldc=256, scales=A,
             lds=4, codes_t=A, ldct=16, scales_t=A, ldst=256)
    a.update(kw)
    return mx.mx_quantize128(*a.values(), 0)


@pytest.mark.parametrize("change,status", [
    (dict(format=0), UNSUPPORTED), (dict(format=3), UNSUPPORTED), (dict(format=-1), UNSUPPORTED),
    (dict(dtype=3), UNSUPPORTED), (dict(dtype=-1), UNSUPPORTED), (dict(flags=1), UNSUPPORTED),
    (dict(flags=1 << 12), UNSUPPORTED),
    (dict(rows=-1), INVALID), (dict(cols=-1), INVALID), (dict(rows=1 << 31), INVALID),
    (dict(cols=1 << 31), INVALID), (dict(rows=1 << 30, cols=1 << 30), INVALID),
    (dict(rows=1 << 21, cols=1 << 19, ldx=1 << 19), SHAPE),   # valid size, short pitches
    (dict(x=None), INVALID), (dict(codes=None, codes_t=None), INVALID),
    (dict(scales=None), INVALID), (dict(scales_t=None), INVALID),
    (dict(ldx=255), SHAPE), (dict(ldc=240), SHAPE), (dict(ldc=264), SHAPE), (dict(cols=250, ldc=250), SHAPE),
    (dict(lds=3), SHAPE), (dict(lds=6), SHAPE), (dict(rows=5, lds=4), SHAPE),
    (dict(ldct=8), SHAPE), (dict(rows=17, lds=20, ldct=16), SHAPE), (dict(ldst=252), SHAPE),
    (dict(x=A + 1), ALIGN), (dict(x=A + 2, dtype=FP32), ALIGN), (dict(codes=A + 8), ALIGN),
    (dict(codes_t=A + 8), ALIGN), (dict(scales=A + 4), ALIGN), (dict(scales_t=A + 8), ALIGN),
    (dict(scales=A + 2, flags=BLOCK), ALIGN),
    (dict(rows=0, x=None, codes=None, codes_t=None), OK), (dict(cols=0, x=None), OK),
])
def test_quantize_refuses(mx, change, status):
    assert quant(mx, **change) == status


def norm(mx, **kw):
    a = dict(x=A, ldx=256, residual=A, weight=A, dtype=BF16, rows=4, cols=256, eps=1e-6, format=E4M3,
             flags=0, h=A, y=A, codes=A, ldc=256, scales=A, lds=4)
    a.update(kw)
    return mx.mx_rms_norm_quant128(*a.values(), 0)


@pytest.mark.parametrize("change,status", [
    (dict(format=5), UNSUPPORTED), (dict(dtype=3), UNSUPPORTED), (dict(flags=BLOCK), UNSUPPORTED),
    (dict(rows=-1), INVALID), (dict(cols=1 << 31), INVALID), (dict(x=None), INVALID),
    (dict(weight=None), INVALID), (dict(codes=None), INVALID), (dict(scales=None), INVALID),
    (dict(eps=-1.0), INVALID), (dict(eps=float("nan")), INVALID),
    (dict(ldx=128), SHAPE), (dict(ldc=128), SHAPE), (dict(ldc=257), SHAPE), (dict(lds=2), SHAPE),
    (dict(x=A + 1), ALIGN), (dict(residual=A + 1), ALIGN), (dict(weight=A + 2, dtype=FP32), ALIGN),
    (dict(h=A + 1), ALIGN), (dict(y=A + 1), ALIGN), (dict(codes=A + 4), ALIGN), (dict(scales=A + 4), ALIGN),
    (dict(rows=0, x=None), OK), (dict(cols=0, x=None), OK),
])
def test_norm_refuses(mx, change, status):
    assert norm(mx, **change) == status


def norm_bwd(mx, **kw):
    a = dict(grad_y=A, h=A, weight=A, gres=A, dtype=BF16, rows=4, cols=256, eps=1e-6, gh=A, gw=A, work=A)
    a.update(kw)
    return mx.mx_rms_norm_bwd(*a.values(), 0)


@pytest.mark.parametrize("change,status", [
    (dict(dtype=4), UNSUPPORTED), (dict(rows=-1), INVALID), (dict(cols=-1), INVALID),
    (dict(grad_y=None), INVALID), (dict(h=None), INVALID), (dict(weight=None), INVALID),
    (dict(gh=None), INVALID), (dict(gw=None), INVALID), (dict(work=None), INVALID), (dict(eps=-1.0), INVALID),
    (dict(grad_y=A + 1), ALIGN), (dict(h=A + 2, dtype=FP32), ALIGN), (dict(gres=A + 1), ALIGN),
    (dict(gh=A + 1), ALIGN), (dict(gw=A + 2), ALIGN), (dict(work=A + 4), ALIGN),
    (dict(cols=0, gw=None), OK),
])
def test_norm_gradient_refuses(mx, change, status):
    assert norm_bwd(mx, **change) == status


def test_norm_gradient_workspace(mx):
    f = mx.mx_rms_norm_bwd_workspace
    assert f(0, 256) == 0 and f(1, 256) == 1024 and f(10, 7) == 640
    assert f(1 << 20, 256) == f(1 << 30, 256) and f(-1, 4) == -1 and f(4, -1) == -1 and f(1 << 31, 1) == -1


def gemm(mx, **kw):
    a = dict(a=A, lda=256, sa=A, ldsa=8, fa=E4M3, b=A, ldb=256, sb=A, ldsb=132, fb=E4M3, flags=0, M=5, N=130,
             K=250, out_fp32=0, d=A, status=A)
    a.update(kw)
    return mx.mx_gemm128(*a.values(), 0)


@pytest.mark.parametrize("change,status", [
    (dict(fa=0), UNSUPPORTED), (dict(fb=7), UNSUPPORTED), (dict(flags=POW2), UNSUPPORTED),
    (dict(out_fp32=2), INVALID), (dict(M=-1), INVALID), (dict(N=-1), INVALID), (dict(K=-1), INVALID),
    (dict(M=1 << 31), INVALID), (dict(M=1 << 30, N=1 << 30), INVALID), (dict(d=None), INVALID),
    (dict(a=None), INVALID), (dict(b=None), INVALID), (dict(sa=None), INVALID), (dict(sb=None), INVALID),
    (dict(sb=None, flags=BLOCK), INVALID),
    (dict(lda=240), SHAPE), (dict(lda=250), SHAPE), (dict(ldb=264), SHAPE), (dict(ldsa=4), SHAPE),
    (dict(ldsa=9), SHAPE), (dict(ldsb=128), SHAPE),
    (dict(a=A + 8), ALIGN), (dict(b=A + 8), ALIGN), (dict(sa=A + 4), ALIGN), (dict(sb=A + 8), ALIGN),
    (dict(sb=A + 2, flags=BLOCK), ALIGN), (dict(d=A + 8), ALIGN), (dict(status=A + 2), ALIGN),
    (dict(M=0, a=None), OK), (dict(N=0, d=None), OK),
])
def test_gemm_refuses(mx, change, status):
    assert gemm(mx, **change) == status


# --------------------------------------------------------- the tensor layer --
# (device checks come first: CPU tensors are refused by name)

def test_tensor_layer_refuses_host_tensors(mx):
    x, w = torch.zeros(4, 256), torch.zeros(256)
    codes, scales = torch.zeros(4, 256, dtype=torch.uint8), torch.zeros(4, 2)
    for call in (lambda: mx.quantize128(x), lambda: mx.rms_norm_quantize(x, w),
                 lambda: mx.rms_norm_bwd(x, x, w), lambda: mx.gemm128(codes, scales, codes, scales),
                 lambda: mx.linear128(x, x), lambda: mx.rms_norm_linear128(x, w, x)):
        with pytest.raises(ValueError, match="CUDA"):
            call()
