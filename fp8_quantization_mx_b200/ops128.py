"""FP8 with one float32 scale per 128 elements: the tensor layer.

``quantize128``, ``rms_norm_quantize`` and ``gemm128`` run one after the other
in a linear layer's forward pass; ``gemm128`` on transposed operands and
``rms_norm_bwd`` are its backward pass. ``linear128`` and
``rms_norm_linear128`` are both passes as autograd functions. See
``include/mx.h`` for the exact arithmetic and layouts.

An operand is a pair ``(codes, scales)``: codes uint8 ``[rows, cols]`` whose
rows are a multiple of 16 bytes apart; scales float32 ``[rows, ceil(cols/128)]``
stored tile-major (strides ``(1, pitch)``), or per 128 x 128 block, contiguous
``[ceil(rows/128), ceil(cols/128)]``.
"""

from __future__ import annotations

import contextlib
import ctypes

import torch

import fp8_quantization_mx_b200 as _c

from . import BLOCK128, E4M3, E5M2, POW2_SCALES

_DTYPES = {torch.bfloat16: 0, torch.float16: 1, torch.float32: 2}
_DIRECTIONS = {"rows": 1, "cols": 2, "both": 3}
_NO_SWITCH = contextlib.nullcontext()


def _on(device):
    """Makes ``device`` current, without the cost of a switch where it is."""
    return _NO_SWITCH if torch.cuda.current_device() == device.index else torch.cuda.device(device)


# Calls with nothing unusual about them go through a C++ module that makes the
# same checks, tensors and C calls (csrc/mx_fast128.cpp); it leaves every other
# call to the code below. None until first used, False where it was not built
# (or for another torch or Python).
_fast = None


def _bind_fast():
    global _fast
    lib = _c.load_library()
    try:
        from . import _fast128
    except ImportError:
        _fast = False
        return False
    _fast128.bind(*(ctypes.cast(f, ctypes.c_void_p).value for f in (
        lib.mx_quantize128, lib.mx_rms_norm_quant128, lib.mx_rms_norm_bwd,
        lib.mx_rms_norm_bwd_workspace, lib.mx_gemm128)))
    _fast = _fast128
    return _fast


def _made(result, where: str) -> bool:
    """Whether the C++ module made the call (raises if the library refused it)."""
    if type(result) is int:
        _c._check(result, where)
    return result is not None


# The current stream's handle by device index, without building a Stream object
# (2 us of a call that takes 10).
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream(device) -> int:
    if _raw_stream is not None:
        return _raw_stream(device.index)
    return torch.cuda.current_stream(device).cuda_stream


def _fp8_format(format, name="format"):
    if format not in (E4M3, E5M2):
        raise ValueError(f"{name} must be E4M3 or E5M2")


def _stored(t, name: str):
    """Refuses a view that torch negates where it reads it: kernels read memory."""
    if t.is_neg():
        raise ValueError(f"{name} must not be lazily negated (use its resolve_neg())")


def _matrix(t, name: str, device=None, dtype=None, shape=None):
    """Checks a 2-D CUDA tensor of a floating type whose rows are contiguous;
    returns its row pitch in elements."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if device is not None and t.device != device:
        raise ValueError(f"{name} must be on {device}, got {t.device}")
    if t.dtype not in _DTYPES:
        raise ValueError(f"{name} must be bfloat16, float16 or float32, got {t.dtype}")
    if dtype is not None and t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if t.dim() != 2:
        raise ValueError(f"{name} must be [rows, cols]")
    rows, cols = t.shape
    if shape is not None and (rows, cols) != shape:
        raise ValueError(f"{name} must be {list(shape)}, got {list(t.shape)}")
    if rows == 0 or cols == 0:
        return cols
    if cols > 1 and t.stride(1) != 1:
        raise ValueError(f"{name} must have contiguous rows")
    if rows > 1 and t.stride(0) < cols:
        raise ValueError(f"{name} must not have overlapping rows")
    _stored(t, name)
    return t.stride(0) if rows > 1 else cols


def _contiguous(t, name: str, device, dtype, shape):
    if not isinstance(t, torch.Tensor) or t.device != device:
        raise ValueError(f"{name} must be a tensor on {device}")
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} must be {list(shape)}, got {list(t.shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    _stored(t, name)


def _new_codes(rows: int, cols: int, device):
    """A code matrix for the quantizers to write, and its row pitch."""
    pitch = (cols + 15) // 16 * 16
    held = torch.empty((rows, pitch), dtype=torch.uint8, device=device)
    return (held if pitch == cols else held[:, :cols]), pitch


def _new_scales(rows: int, cols: int, block: bool, device):
    """Scales for the quantizers to write, and the pitch of tile scales."""
    nb = (cols + 127) // 128
    if block:
        return torch.empty(((rows + 127) // 128, nb), dtype=torch.float32, device=device), 4
    pitch = (rows + 3) // 4 * 4
    held = torch.empty_strided((pitch, nb), (1, pitch), dtype=torch.float32, device=device)
    return (held if pitch == rows else held[:rows]), pitch


def _codes(t, name: str, device, rows=None, cols=None) -> int:
    """Checks a code matrix; returns its row pitch. The bytes of a row up to
    its length rounded up to 16 must lie in the tensor's storage."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.device != device:
        raise ValueError(f"{name} must be on {device}, got {t.device}")
    if t.dtype != torch.uint8:
        raise ValueError(f"{name} must be uint8, got {t.dtype}")
    shape = t.shape
    if len(shape) != 2 or (rows is not None and shape[0] != rows) or \
            (cols is not None and shape[1] != cols):
        raise ValueError(f"{name} must be [{'rows' if rows is None else rows}, "
                         f"{'cols' if cols is None else cols}], got {list(shape)}")
    rows, cols = shape
    need = (cols + 15) // 16 * 16
    if rows == 0 or cols == 0:
        return need
    stride = t.stride()
    pitch = stride[0] if rows > 1 else need
    if pitch == cols == need and stride[1] == 1:
        return pitch   # whole rows end to end: nothing beyond them is read
    if (cols > 1 and stride[1] != 1) or pitch < need or pitch % 16:
        raise ValueError(f"{name} must have contiguous rows a multiple of 16 bytes apart, at least "
                         f"{need}")
    if t.storage_offset() + (rows - 1) * pitch + need > t.untyped_storage().nbytes():
        raise ValueError(f"{name}: the last row's padding to 16 bytes lies outside its storage")
    return pitch


def _scales(t, name: str, device, rows: int, cols: int, block: bool) -> int:
    """Checks the scales of a [rows, cols] operand; returns the pitch of tile
    scales (floats from a tile's scales to the next tile's)."""
    nb = (cols + 127) // 128
    if not isinstance(t, torch.Tensor) or t.device != device:
        raise ValueError(f"{name} must be a tensor on {device}")
    if t.dtype != torch.float32:
        raise ValueError(f"{name} must be float32, got {t.dtype}")
    shape = ((rows + 127) // 128 if block else rows, nb)
    if t.shape != shape:
        raise ValueError(f"{name} must be {list(shape)}, got {list(t.shape)}")
    _stored(t, name)
    if block:
        if not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous")
        return 4
    need = (rows + 3) // 4 * 4
    if rows == 0 or cols == 0:
        return need
    stride = t.stride()
    pitch = stride[1] if nb > 1 else need
    if pitch == need == rows and stride[0] == 1:
        return pitch
    if (rows > 1 and stride[0] != 1) or pitch < need or pitch % 4:
        raise ValueError(f"{name} must be stored tile by tile (strides (1, pitch), pitch a multiple "
                         f"of 4 and at least {need}), as quantize128 returns them")
    if (t.storage_offset() + (nb - 1) * pitch + need) * 4 > t.untyped_storage().nbytes():
        raise ValueError(f"{name}: the last tile's scales, padded to 4, lie outside the storage")
    return pitch


def quantize128(x: torch.Tensor, format: int = E4M3, block: bool = False, direction: str = "rows",
                pow2: bool = False, out=None):
    """FP8-quantizes ``x`` [rows, cols] (bfloat16, float16 or float32; rows may
    be strided) with one float32 scale per 1 x 128 tile, or with ``block`` per
    128 x 128 block. ``direction``:

    * ``"rows"``: ``(codes [rows, cols], scales)``, tiles along the rows;
    * ``"cols"``: ``(codes_t [cols, rows], scales_t)``, the same of x transposed;
    * ``"both"``: ``(codes, scales, codes_t, scales_t)``, from one read of x.

    ``pow2``: power-of-two scales. ``out`` may supply the two or four tensors;
    a row of its codes is written up to a multiple of 16 bytes, a tile's scales
    up to a multiple of 4 rows."""
    _fp8_format(format)
    if direction not in _DIRECTIONS:
        raise ValueError("direction must be 'rows', 'cols' or 'both'")
    if out is None and (_fast or (_fast is None and _bind_fast())):
        r = _fast.quantize(x, format, bool(block), _DIRECTIONS[direction], bool(pow2))
        if _made(r, "mx_quantize128"):
            return r
    ldx = _matrix(x, "x")
    rows, cols = x.shape
    dev = x.device
    sides = (((rows, cols),) if direction != "cols" else ()) + \
            (((cols, rows),) if direction != "rows" else ())
    args, given = [], out
    if out is None:
        out = ()
        for r, c in sides:
            codes, ld = _new_codes(r, c, dev)
            scales, lds = _new_scales(r, c, block, dev)
            out += (codes, scales)
            args += [codes.data_ptr(), ld, scales.data_ptr(), lds]
    elif len(out) != 2 * len(sides):
        raise ValueError(f"out must hold {2 * len(sides)} tensors")
    for i, (r, c) in enumerate(sides if given is not None else ()):
        codes, scales = out[2 * i], out[2 * i + 1]
        ld = _codes(codes, f"out[{2 * i}]", dev, r, c)
        lds = _scales(scales, f"out[{2 * i + 1}]", dev, r, c, block)
        args += [codes.data_ptr(), ld, scales.data_ptr(), lds]
    none = [None, 0, None, 0]
    if direction == "rows":
        args += none
    elif direction == "cols":
        args = none + args
    flags = (BLOCK128 if block else 0) | (POW2_SCALES if pow2 else 0)
    with _on(dev):
        _c._check(_c.mx_quantize128(x.data_ptr(), _DTYPES[x.dtype], rows, cols, ldx, format, flags,
                                   *args, _stream(dev)), "mx_quantize128")
    return tuple(out)


def rms_norm_quantize(x: torch.Tensor, weight: torch.Tensor, residual=None, eps: float = 1e-6,
                      format: int = E4M3, pow2: bool = False, return_y: bool = False, h_out=None,
                      out=None):
    """RMSNorm with the residual's addition and FP8 output, one kernel:
    h = x + residual, y = h * weight / sqrt(mean(h^2) + eps), codes and tile
    scales of y. x [rows, cols] (rows may be strided), residual alike
    (contiguous), weight [cols], all of one type. Returns ``(codes, scales, h,
    y)``: h is None without a residual, y None unless ``return_y``. ``h_out``
    may be a buffer for h (``residual`` itself: in place), ``out`` the two
    buffers of codes and scales."""
    _fp8_format(format)
    if out is None and h_out is None and (_fast or (_fast is None and _bind_fast())):
        r = _fast.norm(x, weight, residual, eps, format, bool(pow2), bool(return_y))
        if _made(r, "mx_rms_norm_quant128"):
            return r
    ldx = _matrix(x, "x")
    rows, cols = x.shape
    dev, dt = x.device, x.dtype
    _contiguous(weight, "weight", dev, dt, (cols,))
    h = y = None
    if residual is not None:
        _contiguous(residual, "residual", dev, dt, (rows, cols))
        h = torch.empty((rows, cols), dtype=dt, device=dev) if h_out is None else h_out
    elif h_out is not None:
        raise ValueError("h_out without a residual: h is x")
    if h_out is not None:
        _contiguous(h_out, "h_out", dev, dt, (rows, cols))
    if return_y:
        y = torch.empty(rows, cols, dtype=dt, device=dev)
    if out is None:
        codes, ld = _new_codes(rows, cols, dev)
        scales, lds = _new_scales(rows, cols, False, dev)
    elif len(out) != 2:
        raise ValueError("out must be (codes, scales)")
    else:
        codes, scales = out
        ld = _codes(codes, "codes", dev, rows, cols)
        lds = _scales(scales, "scales", dev, rows, cols, False)
    with _on(dev):
        _c._check(_c.mx_rms_norm_quant128(
            x.data_ptr(), ldx, None if residual is None else residual.data_ptr(), weight.data_ptr(),
            _DTYPES[dt], rows, cols, eps, format, POW2_SCALES if pow2 else 0,
            None if h is None else h.data_ptr(), None if y is None else y.data_ptr(),
            codes.data_ptr(), ld, scales.data_ptr(), lds, _stream(dev)), "mx_rms_norm_quant128")
    return codes, scales, h, y


def rms_norm_bwd(grad_y: torch.Tensor, h: torch.Tensor, weight: torch.Tensor, eps: float = 1e-6,
                 grad_residual=None, out=None):
    """The gradient of ``rms_norm_quantize``, straight through the quantizer:
    ``(grad_h, grad_weight)`` from grad_y = dL/dy and h (x without a residual).
    grad_h [rows, cols] in h's type is the gradient of x and residual alike;
    ``grad_residual`` (what reaches h from elsewhere) is added to it.
    grad_weight is float32. ``out`` may be a buffer for grad_h (``grad_y`` or
    ``grad_residual`` itself: in place)."""
    if out is None and (_fast or (_fast is None and _bind_fast())):
        r = _fast.norm_bwd(grad_y, h, weight, eps, grad_residual)
        if _made(r, "mx_rms_norm_bwd"):
            return r
    _matrix(h, "h")
    rows, cols = h.shape
    dev, dt = h.device, h.dtype
    for name, t in (("h", h), ("grad_y", grad_y), ("grad_residual", grad_residual), ("out", out)):
        if t is not None:
            _contiguous(t, name, dev, dt, (rows, cols))
        elif name == "grad_y":
            raise ValueError("grad_y must be a tensor")
    _contiguous(weight, "weight", dev, dt, (cols,))
    gh = torch.empty_like(h) if out is None else out
    gw = torch.empty(cols, dtype=torch.float32, device=dev)
    with _on(dev):
        work = torch.empty(_c.mx_rms_norm_bwd_workspace(rows, cols), dtype=torch.uint8, device=dev)
        _c._check(_c.mx_rms_norm_bwd(
            grad_y.data_ptr(), h.data_ptr(), weight.data_ptr(),
            None if grad_residual is None else grad_residual.data_ptr(), _DTYPES[dt], rows, cols, eps,
            gh.data_ptr(), gw.data_ptr(), work.data_ptr(), _stream(dev)), "mx_rms_norm_bwd")
    return gh, gw


def gemm128(a_codes: torch.Tensor, a_scales: torch.Tensor, b_codes: torch.Tensor,
            b_scales: torch.Tensor, a_format: int = E4M3, b_format: int = E4M3,
            out_dtype=torch.bfloat16, out=None, status=None):
    """D [M, N] = A B^T on the tensor cores: A [M, K] with tile scales, B [N, K]
    with tile or block scales (by the shape of ``b_scales``). The product of a
    K-block's two scales has to lie in float32's normal range. bf16 or float32
    out; ``status``: an optional int32 device tensor set nonzero if one of the
    kernel's waits timed out (after a second, which nothing but a device held up
    from outside takes). What of D was left unmade then is NaN, with or without a
    status."""
    _fp8_format(a_format, "a_format")
    _fp8_format(b_format, "b_format")
    if out_dtype not in (torch.bfloat16, torch.float32):
        raise ValueError("out_dtype must be bfloat16 or float32")
    if out is None and status is None and (_fast or (_fast is None and _bind_fast())):
        r = _fast.gemm(a_codes, a_scales, b_codes, b_scales, a_format, b_format,
                       out_dtype == torch.float32)
        if _made(r, "mx_gemm128"):
            return r
    if not isinstance(a_codes, torch.Tensor) or not a_codes.is_cuda:
        raise ValueError("a_codes must be a CUDA tensor")
    dev = a_codes.device
    lda = _codes(a_codes, "a_codes", dev)
    M, K = a_codes.shape
    ldb = _codes(b_codes, "b_codes", dev, cols=K)
    N = b_codes.shape[0]
    ldsa = _scales(a_scales, "a_scales", dev, M, K, False)
    if not isinstance(b_scales, torch.Tensor):
        raise ValueError("b_scales must be a tensor")
    # one row: a tile is a block, and contiguous scales are a block's layout
    block = b_scales.dim() == 2 and b_scales.shape[0] == (N + 127) // 128 and \
        (N > 1 or b_scales.is_contiguous())
    ldsb = _scales(b_scales, "b_scales", dev, N, K, block)
    if out is None:
        out = torch.empty(M, N, dtype=out_dtype, device=dev)
    else:
        _contiguous(out, "out", dev, out_dtype, (M, N))
    if status is not None:
        if not isinstance(status, torch.Tensor) or status.device != dev or \
                status.dtype != torch.int32 or status.numel() < 1:
            raise ValueError(f"status must be an int32 tensor on {dev}")
    with _on(dev):
        _c._check(_c.mx_gemm128(a_codes.data_ptr(), lda, a_scales.data_ptr(), ldsa, a_format,
                               b_codes.data_ptr(), ldb, b_scales.data_ptr(), ldsb, b_format,
                               BLOCK128 if block else 0, M, N, K, int(out_dtype == torch.float32),
                               out.data_ptr(), None if status is None else status.data_ptr(),
                               _stream(dev)), "mx_gemm128")
    return out


# ---------------------------------------------------------------- autograd --

class FP8Linear128(torch.autograd.Function):
    """y = x weight^T in FP8: x and the output's gradient in 1 x 128 tiles along
    each product's sum, the weight in 128 x 128 blocks. x [tokens, K], weight
    [N, K], both bfloat16; gradients come back in bfloat16 and the weight's
    type. The quantizers pass gradients straight through."""

    @staticmethod
    def forward(ctx, x, weight, grad_format=E4M3):
        need_x, need_w = ctx.needs_input_grad[:2]
        x = x.contiguous()
        xq = quantize128(x, direction="both" if need_w else "rows")
        wq = quantize128(weight.contiguous(), block=True, direction="both" if need_x else "rows")
        ctx.grad_format = grad_format
        ctx.save_for_backward(*(xq[2:] if need_w else (None, None)),
                              *(wq[2:] if need_x else (None, None)))
        ctx.weight_dtype = weight.dtype
        return gemm128(xq[0], xq[1], wq[0], wq[1])

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, grad):
        return (*_linear_grads(ctx.saved_tensors, grad, ctx.grad_format, ctx.weight_dtype), None)


def _linear_grads(saved, grad, fmt, weight_dtype):
    """(input gradient, weight gradient), each None where its operand was not kept."""
    xt, xts, wt, wts = saved
    if xt is None and wt is None:
        return None, None
    direction = "both" if xt is not None and wt is not None else "rows" if xt is None else "cols"
    g = quantize128(grad.contiguous(), fmt, direction=direction)
    gx = gw = None
    if wt is not None:
        gx = gemm128(g[0], g[1], wt, wts, a_format=fmt)
    if xt is not None:
        gw = gemm128(g[-2], g[-1], xt, xts, a_format=fmt, out_dtype=torch.float32).to(weight_dtype)
    return gx, gw


class FP8NormLinear128(torch.autograd.Function):
    """(y weight^T, h) with h = x + residual and y its RMSNorm: the norm hands
    its FP8 codes to the product. x, residual [tokens, K] bfloat16."""

    @staticmethod
    def forward(ctx, x, residual, norm_weight, weight, eps=1e-6, grad_format=E4M3):
        need_h = any(ctx.needs_input_grad[:3])
        need_w = ctx.needs_input_grad[3]
        x = x.contiguous()
        codes, scales, h, y = rms_norm_quantize(x, norm_weight, residual, eps, return_y=need_w)
        wq = quantize128(weight.contiguous(), block=True, direction="both" if need_h else "rows")
        yt = quantize128(y, direction="cols") if need_w else (None, None)
        ctx.save_for_backward(*yt, *(wq[2:] if need_h else (None, None)), x if h is None else h,
                              norm_weight)
        ctx.eps, ctx.grad_format, ctx.weight_dtype = eps, grad_format, weight.dtype
        # (without a residual h is x itself: a copy would be a second output)
        return gemm128(codes, scales, wq[0], wq[1]), h

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, grad, grad_h):
        *saved, h, norm_weight = ctx.saved_tensors
        gy, gw = _linear_grads(saved, grad, ctx.grad_format, ctx.weight_dtype)
        gx = gn = None
        if gy is not None:
            gx, gn = rms_norm_bwd(gy, h, norm_weight, ctx.eps,
                                  grad_residual=None if grad_h is None else grad_h.contiguous())
            gn = gn.to(norm_weight.dtype)
        need_x, need_res = ctx.needs_input_grad[:2]
        # one gradient for both, but in memory of its own for each: a leaf keeps the
        # tensor that it is given and adds to it in place
        gr = None if not need_res else gx.clone() if need_x else gx
        return gx if need_x else None, gr, gn, gw, None, None


def _layer_inputs(**tensors):
    for name, t in tensors.items():
        if not isinstance(t, torch.Tensor) or not t.is_cuda:
            raise ValueError(f"{name} must be a CUDA tensor")
        if t.dtype != torch.bfloat16:
            raise ValueError(f"{name} must be bfloat16, got {t.dtype}")


def linear128(x: torch.Tensor, weight: torch.Tensor, grad_format: int = E4M3) -> torch.Tensor:
    """x weight^T with FP8 operands in all three products of training (see
    ``FP8Linear128``). x bfloat16 [..., K], weight bfloat16 [N, K];
    ``grad_format``: the output gradient's FP8 format."""
    _layer_inputs(x=x, weight=weight)
    _fp8_format(grad_format, "grad_format")
    if not torch.is_grad_enabled():   # nothing is kept for a backward pass
        x, weight = x.detach(), weight.detach()
    y = FP8Linear128.apply(x.reshape(-1, x.shape[-1]), weight, grad_format)
    return y.view(*x.shape[:-1], weight.shape[0])


def rms_norm_linear128(x: torch.Tensor, norm_weight: torch.Tensor, weight: torch.Tensor,
                       residual=None, eps: float = 1e-6, grad_format: int = E4M3):
    """``(y weight^T, h)``: h = x + residual (x itself without one), y =
    RMSNorm(h), the product in FP8 from the norm's own codes. Shapes as
    ``linear128``."""
    _layer_inputs(x=x, norm_weight=norm_weight, weight=weight,
                  **({} if residual is None else {"residual": residual}))
    _fp8_format(grad_format, "grad_format")
    shape = x.shape
    if residual is not None and residual.shape != shape:
        raise ValueError(f"residual must be {list(shape)}, got {list(residual.shape)}")
    if not torch.is_grad_enabled():   # nothing is kept for a backward pass
        x, norm_weight, weight = x.detach(), norm_weight.detach(), weight.detach()
        residual = None if residual is None else residual.detach()
    res = None if residual is None else residual.reshape(-1, shape[-1]).contiguous()
    out, h = FP8NormLinear128.apply(x.reshape(-1, shape[-1]), res, norm_weight, weight, eps,
                                    grad_format)
    return out.view(*shape[:-1], weight.shape[0]), x if h is None else h.view(shape)
