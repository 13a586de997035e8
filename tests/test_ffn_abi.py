"""Host-side checks of the linear layers' and the norm's C ABI and of their
Python entry points (no GPU compute): bad arguments are refused with the
documented status before anything is enqueued.  The addresses are made up and
never followed."""
import math
import os

import pytest
import torch

import fp4_block_scaled_row_amd as fq
from fp4_block_scaled_row_amd import _lib
from test_kv_abi import A, fields

INVALID, UNSUPPORTED, OK, WORKSPACE = (getattr(_lib, "FP4Q_" + s) for s in
                                       ("ERR_INVALID_ARG", "ERR_UNSUPPORTED", "OK", "ERR_WORKSPACE"))


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(_lib.LIB_PATH):
        pytest.skip("libfp4q.so not built (run __graft_entry__.build())")
    return _lib.load()


def weight(**kw):
    w = _lib.WeightArgs()
    return fields(fields(w, format=_lib.FP4Q_NVFP4, n=96, k=128, codes=A, scales=A, global_scale=A), **kw)


def linear_args(**kw):
    a = _lib.LinearArgs()
    fields(a, x=A, rows=4, x_stride=128, x_dtype=_lib.FP4Q_BF16, out_dtype=_lib.FP4Q_BF16, out=A)
    return fields(a, **kw)


def calls(lib):
    return lib.fp4q_linear, lib.fp4q_gated, lib.fp4q_linear_backward


@pytest.mark.parametrize("kw,want", [
    (dict(format=9), INVALID), (dict(format=-1), INVALID), (dict(format=_lib.FP4Q_IF4), UNSUPPORTED),
    (dict(format=_lib.FP4Q_MXFP8), UNSUPPORTED), (dict(n=-2), INVALID), (dict(k=-16), INVALID), (dict(k=24), INVALID),
    (dict(format=_lib.FP4Q_MXFP4, k=48), INVALID), (dict(n=1 << 31), UNSUPPORTED), (dict(k=1 << 31), UNSUPPORTED),
    (dict(codes=None), INVALID), (dict(scales=None), INVALID), (dict(global_scale=None), INVALID),
    (dict(global_scale=A + 2), UNSUPPORTED),
], ids=str)
def test_weights(lib, kw, want):
    for kind, call in enumerate(calls(lib)):
        assert call(weight(**kw), linear_args(), None, 0, None) == want
        assert lib.fp4q_linear_workspace_bytes(weight(**kw), linear_args(), kind) == 0


@pytest.mark.parametrize("kw,want", [
    (dict(rows=-1), INVALID), (dict(rows=1 << 31), UNSUPPORTED), (dict(x_stride=-1), INVALID), (dict(x=None), INVALID),
    (dict(out=None), INVALID), (dict(x_dtype=7), INVALID), (dict(out_dtype=2), INVALID), (dict(out=A + 1), UNSUPPORTED),
    (dict(x=A + 1), UNSUPPORTED), (dict(x=A + 2, x_dtype=_lib.FP4Q_F32), UNSUPPORTED),
    (dict(out=A + 2, out_dtype=_lib.FP4Q_F32), UNSUPPORTED),
], ids=str)
def test_linear_arguments(lib, kw, want):
    for call in calls(lib):
        assert call(weight(), linear_args(**kw), None, 0, None) == want


def test_linear_combinations(lib):
    eight = dict(x_dtype=_lib.FP4Q_E4M3, x_scales=A)
    assert lib.fp4q_linear(weight(), linear_args(**dict(eight, x_scales=None)), None, 0, None) == INVALID
    assert lib.fp4q_linear(weight(), linear_args(**dict(eight, x_stride=160)), None, 0, None) == INVALID
    assert lib.fp4q_linear(weight(k=48), linear_args(**dict(eight, x_stride=48)), None, 0, None) == INVALID
    assert lib.fp4q_linear_backward(weight(), linear_args(**eight), None, 0, None) == UNSUPPORTED
    assert lib.fp4q_gated(weight(n=97), linear_args(), None, 0, None) == INVALID
    assert lib.fp4q_gated(weight(), linear_args(bias=A), None, 0, None) == UNSUPPORTED
    assert lib.fp4q_linear_backward(weight(), linear_args(bias=A), None, 0, None) == UNSUPPORTED
    assert lib.fp4q_linear(weight(), linear_args(products=A), None, 0, None) == UNSUPPORTED
    assert lib.fp4q_gated(weight(), linear_args(products=A, products_dtype=3), None, 0, None) == INVALID
    assert lib.fp4q_gated(weight(), linear_args(products=A + 2), None, 0, None) == UNSUPPORTED
    assert lib.fp4q_linear(weight(), linear_args(bias=A + 1), None, 0, None) == UNSUPPORTED
    assert lib.fp4q_linear(weight(n=1 << 30, k=16), linear_args(rows=1 << 20, x_stride=16), None, 0, None) == UNSUPPORTED
    for call in calls(lib):
        assert call(None, linear_args(), None, 0, None) == INVALID
        assert call(weight(), None, None, 0, None) == INVALID
    assert lib.fp4q_linear_workspace_bytes(weight(), linear_args(), 3) == 0
    assert lib.fp4q_linear_workspace_bytes(None, None, 0) == 0


def test_linear_nothing_to_do(lib):
    for call in calls(lib):
        assert call(weight(), linear_args(rows=0, x=None, out=None), None, 0, None) == OK
    w = weight(n=0, codes=None, scales=None)
    assert lib.fp4q_linear(w, linear_args(), None, 0, None) == OK
    assert lib.fp4q_gated(w, linear_args(), None, 0, None) == OK
    w = weight(k=0, codes=None, scales=None)
    assert lib.fp4q_linear_backward(w, linear_args(), None, 0, None) == OK


def test_linear_workspace(lib):
    """A call whose sums several workgroups share asks for its workspace and refuses a short or misaligned one."""
    w, a = weight(n=256, k=1 << 16), linear_args(rows=128, x_stride=1 << 16)
    need = lib.fp4q_linear_workspace_bytes(w, a, _lib.FP4Q_LINEAR)
    assert need > 0 and need % (128 * 256 * 4) == 0
    for ws, size in ((None, need), (A, need - 1), (A + 8, need)):
        assert lib.fp4q_linear(w, a, ws, size, None) == WORKSPACE


def grad_args(**kw):
    a = _lib.GatedGradArgs()
    return fields(fields(a, dh=A, products=A, dproducts=A, rows=4, f=40, dh_stride=40, dtype=_lib.FP4Q_BF16,
                         products_dtype=_lib.FP4Q_BF16), **kw)


@pytest.mark.parametrize("kw,want", [
    (dict(rows=-1), INVALID), (dict(f=-1), INVALID), (dict(dh_stride=-1), INVALID), (dict(dtype=2), INVALID),
    (dict(products_dtype=5), INVALID), (dict(dh=None), INVALID), (dict(products=None), INVALID),
    (dict(dproducts=None), INVALID), (dict(dh=A + 1), UNSUPPORTED), (dict(dproducts=A + 1), UNSUPPORTED),
    (dict(products=A + 2, products_dtype=_lib.FP4Q_F32), UNSUPPORTED), (dict(products_dtype=_lib.FP4Q_F32), INVALID),
    (dict(rows=1 << 31), UNSUPPORTED), (dict(f=1 << 30), UNSUPPORTED), (dict(rows=1 << 30, f=1 << 20), UNSUPPORTED),
], ids=str)
def test_gated_grad(lib, kw, want):
    assert lib.fp4q_gated_grad(grad_args(**kw), None) == want
    assert lib.fp4q_gated_grad(None, None) == INVALID
    assert lib.fp4q_gated_grad(grad_args(rows=0), None) == OK
    assert lib.fp4q_gated_grad(grad_args(f=0), None) == OK


def norm_args(**kw):
    a = _lib.RmsNormArgs()
    return fields(fields(a, x=A, x_stride=64, weight=A, y=A, rows=4, d=64, dtype=_lib.FP4Q_BF16,
                         weight_dtype=_lib.FP4Q_BF16, eps=1e-6), **kw)


@pytest.mark.parametrize("kw,want", [
    (dict(rows=-1), INVALID), (dict(d=-1), INVALID), (dict(x_stride=-1), INVALID), (dict(residual_stride=-1), INVALID),
    (dict(dtype=2), INVALID), (dict(weight_dtype=7), INVALID), (dict(eps=-1e-6), INVALID), (dict(eps=math.inf), INVALID),
    (dict(eps=math.nan), INVALID), (dict(x=None), INVALID), (dict(weight=None), INVALID), (dict(y=None), INVALID),
    (dict(residual=A), INVALID), (dict(summed=A), INVALID), (dict(codes=A), INVALID), (dict(scales=A), INVALID),
    (dict(codes=A, scales=A), UNSUPPORTED), (dict(codes=A, scales=A, y=None, d=48), INVALID), (dict(d=32769), UNSUPPORTED),
    (dict(rows=1 << 31), UNSUPPORTED), (dict(x=A + 1), UNSUPPORTED), (dict(y=A + 1), UNSUPPORTED),
    (dict(weight=A + 2, weight_dtype=_lib.FP4Q_F32), UNSUPPORTED), (dict(rstd=A + 2), UNSUPPORTED),
], ids=str)
def test_norm(lib, kw, want):
    assert lib.fp4q_rms_norm(norm_args(**kw), None) == want
    assert lib.fp4q_rms_norm(None, None) == INVALID
    assert lib.fp4q_rms_norm(norm_args(rows=0, x=None, y=None), None) == OK


def norm_grad_args(**kw):
    a = _lib.RmsNormGradArgs()
    return fields(fields(a, dy=A, s=A, dy_stride=64, s_stride=64, weight=A, rstd=A, dx=A, dw=A, rows=4, d=64,
                         dtype=_lib.FP4Q_BF16, weight_dtype=_lib.FP4Q_BF16), **kw)


@pytest.mark.parametrize("kw,want", [
    (dict(rows=-1), INVALID), (dict(d=-1), INVALID), (dict(dy_stride=-1), INVALID), (dict(s_stride=-1), INVALID),
    (dict(ds_stride=-1), INVALID), (dict(dtype=2), INVALID), (dict(weight_dtype=-1), INVALID), (dict(dy=None), INVALID),
    (dict(s=None), INVALID), (dict(weight=None), INVALID), (dict(rstd=None), INVALID), (dict(dx=None), INVALID),
    (dict(dw=None), INVALID), (dict(d=32769), UNSUPPORTED), (dict(rows=1 << 31), UNSUPPORTED), (dict(dx=A + 1), UNSUPPORTED),
    (dict(ds=A + 1), UNSUPPORTED), (dict(rstd=A + 1), UNSUPPORTED),
], ids=str)
def test_norm_backward(lib, kw, want):
    assert lib.fp4q_rms_norm_backward(norm_grad_args(**kw), A, 1 << 40, None) == want
    assert lib.fp4q_rms_norm_backward_workspace_bytes(norm_grad_args(**kw)) == 0


def test_norm_backward_workspace(lib):
    a = norm_grad_args()
    need = lib.fp4q_rms_norm_backward_workspace_bytes(a)
    assert need == 4 * 64 * 4           # a part for each row, where there are few
    for ws, size in ((None, need), (A, need - 1), (A + 8, need)):
        assert lib.fp4q_rms_norm_backward(a, ws, size, None) == WORKSPACE
    assert lib.fp4q_rms_norm_backward(norm_grad_args(d=0), None, 0, None) == OK


def test_dequantize_mxfp8(lib):
    assert lib.fp4q_dequantize(_lib.FP4Q_MXFP8, 4, 64, 16, A, A, None, 0, A, None) == UNSUPPORTED
    assert lib.fp4q_dequantize(_lib.FP4Q_MXFP8, 4, 48, 32, A, A, None, 0, A, None) == INVALID
    assert lib.fp4q_dequantize(_lib.FP4Q_MXFP8, 4, 64, 32, A + 2, A, None, 0, A, None) == UNSUPPORTED
    assert lib.fp4q_dequantize(_lib.FP4Q_MXFP8, 0, 64, 32, None, None, None, 0, None, None) == OK


# ---- the Python entry points, as far as they go without a GPU

def test_weight_handle_wants_gpu_planes():
    codes, scales = torch.zeros(4, 16, dtype=torch.uint8), torch.zeros(4, 2, dtype=torch.uint8)
    with pytest.raises(ValueError, match="format"):
        fq.Fp4Weight("if4", codes, scales)
    with pytest.raises(ValueError, match="GPU"):
        fq.Fp4Weight("nvfp4", codes, scales, torch.ones(1))
    with pytest.raises(ValueError, match="GPU"):
        fq.fp4_weight(fq.MxResult(codes, scales, None, None))


def test_calls_want_a_weight_and_gpu_rows():
    x = torch.zeros(2, 32, dtype=torch.bfloat16)
    for call in (fq.fp4_linear, fq.fp4_gated, fq.fp4_linear_backward):
        with pytest.raises(TypeError, match="Fp4Weight"):
            call(x, x)
    with pytest.raises(ValueError, match="GPU"):
        fq.rms_norm(x, torch.ones(32))
    with pytest.raises(ValueError, match="GPU"):
        fq.rms_norm_backward(x, x, torch.ones(32), torch.ones(2))
