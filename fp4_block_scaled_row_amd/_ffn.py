"""Linear layers over 4-bit weights and the norm in front of them: a
feed-forward block whose weights stay as quantize_mxfp4 / quantize_nvfp4 wrote
them, forward and backward (the binding of fp4q_linear, fp4q_gated,
fp4q_rms_norm and their backward calls of include/fp4q.h).

Activations are bf16, fp32, or MXFP8 (Mx8Result, as rms_norm writes it): E4M3
codes with one power-of-two scale for each 32.  Weights and activations enter
the products exactly, sums are fp32, results are rounded once.

One exception: MXFP8 activations with MXFP4 weights, many rows and results in bf16
alone go through the block-scaled matrix instructions, whose sums of eight
neighbouring products may lose what lies below 2^-13 of the largest of them (over a
whole output that is below bf16's rounding).  Who wants fp32 sums there asks for
out_dtype=torch.float32.

The same call on the same tensors gives the same bits each time.  Which kernel a
call takes, and so the order of its sums, goes by shapes, types, x's row stride, the
alignment of the planes, and whether products are asked for and in which type.

As everywhere in this package, calls record no gradients: results require none,
whatever the arguments do.  A training program joins a forward and a backward call in
an autograd.Function of its own:

    class Linear(torch.autograd.Function):
        @staticmethod
        def forward(ctx, x, w):
            ctx.w = w
            return fp4_linear(x, w)

        @staticmethod
        def backward(ctx, dy):
            return fp4_linear_backward(dy.contiguous(), ctx.w), None
"""
from collections import namedtuple

import torch

from . import _lib
from ._kv import _raw_stream

__all__ = ["Fp4Weight", "fp4_weight", "fp4_linear", "fp4_linear_backward", "fp4_gated", "fp4_gated_backward",
           "Mx8Result", "NormResult", "rms_norm", "rms_norm_backward"]

#: MXFP8 rows: codes [rows, cols] uint8 (E4M3), scales [rows, cols / 32] uint8 (E8M0).
Mx8Result = namedtuple("Mx8Result", "codes scales")
NormResult = namedtuple("NormResult", "out summed rstd")

_FORMATS = {"nvfp4": (_lib.FP4Q_NVFP4, 16), "mxfp4": (_lib.FP4Q_MXFP4, 32)}
_DTYPES = {torch.float32: _lib.FP4Q_F32, torch.bfloat16: _lib.FP4Q_BF16}


def _call(index, function, *args):
    """function(*args) with device `index` as the current one."""
    if torch.cuda.current_device() == index:
        return function(*args)
    with torch.cuda.device(index):
        return function(*args)


class Fp4Weight:
    """A weight [n, k] over planes that the caller owns.  Checked once, here;
    the calls below take it as it is.  codes: uint8 [n, k / 2]; scales: uint8
    [n, k / 16] ("nvfp4", with the one float32 of global_scale) or [n, k / 32]
    ("mxfp4")."""

    def __init__(self, format, codes, scales, global_scale=None):
        if format not in _FORMATS:
            raise ValueError("fp4q: a weight's format is 'nvfp4' or 'mxfp4', got %r" % (format,))
        code, block = _FORMATS[format]
        for what, t in (("codes", codes), ("scales", scales)):
            if not isinstance(t, torch.Tensor) or not t.is_cuda or t.dtype != torch.uint8 or t.dim() != 2 \
                    or not t.is_contiguous():
                raise ValueError("fp4q: a weight's %s must be a contiguous 2-D uint8 GPU tensor" % what)
        n, k = codes.shape[0], codes.shape[1] * 2
        if k % block or tuple(scales.shape) != (n, k // block) or scales.device != codes.device:
            raise ValueError("fp4q: inconsistent weight planes: codes %s, scales %s" %
                             (tuple(codes.shape), tuple(scales.shape)))
        if format == "nvfp4":
            if not isinstance(global_scale, torch.Tensor) or global_scale.device != codes.device \
                    or global_scale.dtype != torch.float32 or global_scale.numel() != 1:
                raise ValueError("fp4q: global_scale must be one float32 on the weight's device")
        else:
            global_scale = None
        self.format, self.n, self.k, self.device = format, n, k, codes.device
        # (kept here, so that the addresses stay theirs)
        self.codes, self.scales, self.global_scale = codes, scales, global_scale
        self._args = _lib.WeightArgs(code, n, k, codes.data_ptr(), scales.data_ptr(),
                                     None if global_scale is None else global_scale.data_ptr())
        self._index = codes.get_device()


def fp4_weight(quantized):
    """The Fp4Weight of a quantize_mxfp4 or quantize_nvfp4 result.  One of policy
    "if4" is refused: the products do not take its blocks of integers."""
    if getattr(quantized, "policy", None) == "if4":
        raise ValueError("fp4q: a weight is in NVFP4 or MXFP4; IF4 blocks of integers are not")
    g = getattr(quantized, "global_scale", None)
    return Fp4Weight("mxfp4" if g is None else "nvfp4", quantized.codes, quantized.scales, g)


def _rows(t, what, index, cols):
    """Checks a [rows, cols] tensor of fp32 or bf16 with contiguous rows on device `index`; its rows, row stride and
    dtype code."""
    if not isinstance(t, torch.Tensor) or t.get_device() != index or index < 0:
        raise ValueError("fp4q: %s must be a GPU tensor on the other operands' device" % what)
    code = _DTYPES.get(t.dtype)
    if code is None:
        raise TypeError("fp4q: %s must be float32 or bfloat16, got %s" % (what, t.dtype))
    shape = t.shape
    if len(shape) != 2 or shape[1] != cols:
        raise ValueError("fp4q: %s must be [rows, %d], got %s" % (what, cols, tuple(shape)))
    stride, inner = t.stride()
    if inner != 1 and cols > 1:
        raise ValueError("fp4q: rows of %s must be contiguous (stride(1) == 1)" % what)
    return shape[0], stride, code


def _out_dtype(dtype):
    code = _DTYPES.get(dtype)
    if code is None:
        raise TypeError("fp4q: out_dtype must be float32 or bfloat16, got %s" % dtype)
    return code


def _buffer(t, what, shape, dtype, device, *others):
    """A dense buffer of this shape and dtype: t after checks, apart from the others, or a new one."""
    if t is None:
        return torch.empty(shape, dtype=dtype, device=device)
    if not isinstance(t, torch.Tensor) or t.dtype != dtype or t.shape != shape or t.device != device \
            or not t.is_contiguous():
        raise ValueError("fp4q: %s must be a contiguous %s tensor of shape %s on %s" % (what, dtype, shape, device))
    if others:
        _apart(t, what, *others)
    return t


def _apart(t, what, *others):
    """Refuses a buffer t of the caller's that overlaps one of the others (2-D or dense tensors, or None)."""
    lo, hi = t.data_ptr(), t.data_ptr() + t.numel() * t.element_size()
    for o in others:
        if o is None or o.numel() == 0:
            continue
        span = (sum((n - 1) * s for n, s in zip(o.shape, o.stride())) + 1) * o.element_size()
        if lo < o.data_ptr() + span and o.data_ptr() < hi:
            raise ValueError("fp4q: %s must not overlap what the call reads or its other results" % what)


def _activations(x, w, out_dtype):
    """x of a linear layer as LinearArgs fields, and the output's dtype."""
    if isinstance(x, Mx8Result):
        codes, scales = x
        for what, t, cols in (("x.codes", codes, w.k), ("x.scales", scales, w.k // 32)):
            if not isinstance(t, torch.Tensor) or not t.is_cuda or t.get_device() != w._index \
                    or t.dtype != torch.uint8 or t.dim() != 2 or t.shape[1] != cols or not t.is_contiguous():
                raise ValueError("fp4q: %s must be a contiguous uint8 [rows, %d] tensor on the weight's device" %
                                 (what, cols))
        if w.k % 32 or codes.shape[0] != scales.shape[0]:
            raise ValueError("fp4q: inconsistent MXFP8 planes: codes %s, scales %s" %
                             (tuple(codes.shape), tuple(scales.shape)))
        return codes, (codes.data_ptr(), scales.data_ptr(), codes.shape[0], w.k, _lib.FP4Q_E4M3), \
            torch.bfloat16 if out_dtype is None else out_dtype
    rows, stride, code = _rows(x, "x", w._index, w.k)
    return x, (x.data_ptr(), None, rows, stride, code), x.dtype if out_dtype is None else out_dtype


def _linear(w, a, kind, function, where):
    """Makes the call, with memory for parts of sums where it asks for some: from
    torch's allocator each time, so that calls on other streams and captured ones
    have their own."""
    stream = _raw_stream(w._index)
    status = _call(w._index, function, w._args, a, None, 0, stream)
    if status == _lib.FP4Q_ERR_WORKSPACE:
        need = _call(w._index, _lib.load().fp4q_linear_workspace_bytes, w._args, a, kind)
        ws = torch.empty(need, dtype=torch.uint8, device=w.device)
        status = _call(w._index, function, w._args, a, ws.data_ptr(), need, stream)
    if status:
        _lib.check(status, where)


def _weight(w):
    if not isinstance(w, Fp4Weight):
        raise TypeError("fp4q: the weight must be an Fp4Weight (fp4_weight of a quantized tensor)")
    return w


def fp4_linear(x, w, *, bias=None, out_dtype=None, out=None):
    """x W^T (+ bias): x [rows, k] bf16 or fp32 (any row stride), or an Mx8Result;
    w an Fp4Weight [n, k].

    Returns [rows, n] in out_dtype: x's by default, bf16 for MXFP8 (with an MXFP4
    weight and many rows by sums of fewer bits, see this module; torch.float32 has
    fp32 ones).  bias: [n] of that dtype, added before the one rounding."""
    _weight(w)
    _, fields, dtype = _activations(x, w, out_dtype)
    code = _out_dtype(dtype)
    if bias is not None:
        _buffer(bias, "bias", (w.n,), dtype, w.device)
    out = _buffer(out, "out", (fields[2], w.n), dtype, w.device, *(x if isinstance(x, Mx8Result) else (x,)), bias,
                  w.codes, w.scales, w.global_scale)
    a = _lib.LinearArgs(*fields, code, None if bias is None else bias.data_ptr(), out.data_ptr(), None, code)
    _linear(w, a, _lib.FP4Q_LINEAR, _lib.load().fp4q_linear, "fp4q_linear")
    return out


def fp4_linear_backward(dy, w, *, out=None):
    """dy W: the gradient of fp4_linear's x from that of its result, dy [rows, n]
    bf16 or fp32, rows contiguous.  Returns [rows, k] in dy's dtype.  (The weight is
    frozen; the gradient of a bias is dy.sum(0).)"""
    _weight(w)
    rows, stride, code = _rows(dy, "dy", w._index, w.n)
    out = _buffer(out, "out", (rows, w.k), dy.dtype, w.device, dy, w.codes, w.scales, w.global_scale)
    a = _lib.LinearArgs(dy.data_ptr(), None, rows, stride, code, code, None, out.data_ptr(), None, code)
    _linear(w, a, _lib.FP4Q_LINEAR_BACKWARD, _lib.load().fp4q_linear_backward, "fp4q_linear_backward")
    return out


def fp4_gated(x, w, *, return_products=False, products_dtype=torch.float32, out_dtype=None, out=None):
    """SiLU(x Wg^T) * (x Wu^T) in one pass: w an Fp4Weight [2 f, k] whose first f
    rows are Wg and whose others are Wu; x as for fp4_linear.

    Returns [rows, f], or with return_products (out, products): products [rows,
    2 f], the two products side by side, which fp4_gated_backward takes: the fp32
    sums, or with products_dtype=torch.bfloat16 their rounding, which halves what a
    training step keeps and moves the gradients by it (2^-8 of a product).  With
    MXFP8 x and an MXFP4 weight the call without products, or with bf16 ones, may
    take sums of fewer bits than the one with fp32 products (see this module)."""
    _weight(w)
    if w.n % 2:
        raise ValueError("fp4q: a gated weight has an even number of rows, got %d" % w.n)
    _, fields, dtype = _activations(x, w, out_dtype)
    code = _out_dtype(dtype)
    out = _buffer(out, "out", (fields[2], w.n // 2), dtype, w.device, *(x if isinstance(x, Mx8Result) else (x,)),
                  w.codes, w.scales, w.global_scale)
    products = None
    if return_products:
        products = torch.empty((fields[2], w.n), dtype=products_dtype, device=w.device)
    a = _lib.LinearArgs(*fields, code, None, out.data_ptr(), products.data_ptr() if return_products else None,
                        _out_dtype(products_dtype))
    _linear(w, a, _lib.FP4Q_GATED, _lib.load().fp4q_gated, "fp4q_gated")
    return (out, products) if return_products else out


def fp4_gated_backward(dh, products, w):
    """(dx, dproducts): the gradients of fp4_gated's x, [rows, k], and of its
    products, [rows, 2 f] (what adapters beside the weight need), from that of its
    result, dh [rows, f] bf16 or fp32, and the products that it returned.  Both in
    dh's dtype; dx is that of the returned dproducts: with bf16 ones it has their
    rounding and its own (2.3e-3 of it as a whole, where one is 1.7e-3).  Who wants
    one rounding alone passes dh.float() and rounds dx."""
    _weight(w)
    if w.n % 2:
        raise ValueError("fp4q: a gated weight has an even number of rows, got %d" % w.n)
    rows, stride, code = _rows(dh, "dh", w._index, w.n // 2)
    p_code = _out_dtype(getattr(products, "dtype", None))
    _buffer(products, "products", (rows, w.n), products.dtype, w.device)
    dproducts = torch.empty((rows, w.n), dtype=dh.dtype, device=w.device)
    g = _lib.GatedGradArgs(dh.data_ptr(), products.data_ptr(), dproducts.data_ptr(), rows, w.n // 2, stride, code,
                           p_code)
    status = _call(w._index, _lib.load().fp4q_gated_grad, g, _raw_stream(w._index))
    if status:
        _lib.check(status, "fp4q_gated_grad")
    return fp4_linear_backward(dproducts, w), dproducts


def _vector(t, what, d, index):
    if not isinstance(t, torch.Tensor) or t.get_device() != index or t.shape != (d,) or not t.is_contiguous():
        raise ValueError("fp4q: %s must be a contiguous [%d] tensor on x's device" % (what, d))
    code = _DTYPES.get(t.dtype)
    if code is None:
        raise TypeError("fp4q: %s must be float32 or bfloat16, got %s" % (what, t.dtype))
    return code


def rms_norm(x, weight, *, residual=None, eps=1e-6, quantize=None, return_rstd=False, out=None, summed=None):
    """s = x + residual (rounded to their dtype), y = s / sqrt(mean(s^2) + eps) *
    weight over each row of x, [rows, d] fp32 or bf16, d to 32768; weight [d] fp32
    or bf16.

    Returns NormResult(out, summed, rstd): out is y in x's dtype, or with
    quantize="mxfp8" (d a multiple of 32) an Mx8Result, which fp4_linear and
    fp4_gated take and dequantize("mxfp8", ...) reads; summed is s (None without
    a residual: it is x); rstd, fp32 [rows], with return_rstd, for
    rms_norm_backward.  out, summed: buffers to write; either may be a dense x or
    residual itself (summed so updates a residual stream in place), and overlaps
    nothing else."""
    if not isinstance(x, torch.Tensor) or not x.is_cuda or x.dim() != 2:
        raise ValueError("fp4q: x must be a 2-D GPU tensor")
    index, d, device = x.get_device(), x.shape[1], x.device
    rows, stride, code = _rows(x, "x", index, d)
    w_code = _vector(weight, "weight", d, index)
    r_stride = 0
    given = out is not None or summed is not None
    if residual is not None:
        r_rows, r_stride, r_code = _rows(residual, "residual", index, d)
        if r_rows != rows or r_code != code:
            raise ValueError("fp4q: residual must have x's shape and dtype")
        summed = torch.empty_like(x) if summed is None and x.is_contiguous() else \
            _buffer(summed, "summed", (rows, d), x.dtype, device)
    elif summed is not None:
        raise ValueError("fp4q: without a residual there is no sum to write")
    if quantize is None:
        out = _buffer(out, "out", (rows, d), x.dtype, device)
        y, codes, scales = out.data_ptr(), None, None
    elif quantize == "mxfp8":
        if d % 32:
            raise ValueError("fp4q: MXFP8 rows are multiples of 32, got %d" % d)
        if out is not None and (not isinstance(out, tuple) or len(out) != 2):
            raise ValueError("fp4q: out of an MXFP8 norm is an Mx8Result")
        c, s = (None, None) if out is None else out
        out = Mx8Result(_buffer(c, "out.codes", (rows, d), torch.uint8, device),
                        _buffer(s, "out.scales", (rows, d // 32), torch.uint8, device))
        y, codes, scales = None, out.codes.data_ptr(), out.scales.data_ptr()
    else:
        raise ValueError("fp4q: quantize is None or 'mxfp8', got %r" % (quantize,))
    if given:
        # a row is read before any of it is written: y and s may be written over the whole of x or residual
        results = list(out) if quantize else [out]
        for i, t in enumerate(results + ([] if summed is None else [summed])):
            over = [o for o in (x, residual) if o is not None and not (o.is_contiguous() and o.data_ptr() == t.data_ptr()
                                                                      and t.dtype == o.dtype)]
            _apart(t, "out or summed", weight, *over, *results[i + 1:], *([summed] if i < len(results) else []))
    rstd = torch.empty(rows, dtype=torch.float32, device=device) if return_rstd else None
    a = _lib.RmsNormArgs(x.data_ptr(), None if residual is None else residual.data_ptr(), stride, r_stride,
                         weight.data_ptr(), y, None if summed is None else summed.data_ptr(),
                         None if rstd is None else rstd.data_ptr(), codes, scales, rows, d, code, w_code, float(eps))
    status = _call(index, _lib.load().fp4q_rms_norm, a, _raw_stream(index))
    if status:
        _lib.check(status, "fp4q_rms_norm")
    return NormResult(out, summed, rstd)


def rms_norm_backward(dy, s, weight, rstd, *, dsummed=None):
    """(dx, dweight) of rms_norm: dy [rows, d] is the gradient of y, s the rows
    that were normed (summed, or x without a residual), rstd as returned.  dx, in
    dy's dtype, is the gradient of s, and so of x and of residual alike; dsummed,
    the gradient that reaches s by other ways, is added to it.  dweight is in
    weight's dtype."""
    if not isinstance(dy, torch.Tensor) or not dy.is_cuda or dy.dim() != 2:
        raise ValueError("fp4q: dy must be a 2-D GPU tensor")
    index, d, device = dy.get_device(), dy.shape[1], dy.device
    rows, stride, code = _rows(dy, "dy", index, d)
    strides = [stride, 0, 0]
    for i, (what, t) in enumerate((("s", s), ("dsummed", dsummed))):
        if t is None and i == 1:
            continue
        t_rows, strides[i + 1], t_code = _rows(t, what, index, d)
        if t_rows != rows or t_code != code:
            raise ValueError("fp4q: %s must have dy's shape and dtype" % what)
    w_code = _vector(weight, "weight", d, index)
    _buffer(rstd, "rstd", (rows,), torch.float32, device)
    dx = torch.empty((rows, d), dtype=dy.dtype, device=device)
    dw = torch.empty_like(weight)
    a = _lib.RmsNormGradArgs(dy.data_ptr(), s.data_ptr(), None if dsummed is None else dsummed.data_ptr(), *strides,
                             weight.data_ptr(), rstd.data_ptr(), dx.data_ptr(), dw.data_ptr(), rows, d, code, w_code)
    lib = _lib.load()
    need = _call(index, lib.fp4q_rms_norm_backward_workspace_bytes, a)
    ws = torch.empty(need, dtype=torch.uint8, device=device) if need else None
    status = _call(index, lib.fp4q_rms_norm_backward, a, ws.data_ptr() if need else None, need, _raw_stream(index))
    if status:
        _lib.check(status, "fp4q_rms_norm_backward")
    return dx, dw
