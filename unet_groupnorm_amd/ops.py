"""Torch binding of include/gn_ops.h: the root-mean-square norm over rows with the residual's
addition (forward, backward, 8-bit output) and the norm of many gradients with clipping.

Argument marshalling only, as in gn.py: every function has the name of the C entry point it
calls, the compiled module _gnbind checks the tensors, allocates outputs and workspaces that
are not given on the inputs' device, and calls the library on that device's current stream;
a non-zero status becomes a GnError. All arithmetic happens in the HIP kernels.

A row is the last dimension. x may be a view whose rows are evenly spaced (a slice of a wider
projection); every other tensor is contiguous. Nothing here waits for the GPU. Tensors that
are given to be written count as modified in place for autograd.
"""
import torch
from torch.autograd.function import once_differentiable

from . import _gnbind
from ._lib import GN_OK, JOIN_STATUS_NAMES, OPS_STATUS_NAMES, STATUS_NAMES, lib
from .gn import _DT, GnError, _out_code

_Q = {torch.int8: 0, torch.float8_e4m3fn: 1}
_NORM = {2: 0, 2.0: 0, float("inf"): 1}


def _check(fn, status):
    if status != GN_OK:
        e = GnError(fn, status)
        name = {**OPS_STATUS_NAMES, **JOIN_STATUS_NAMES, **STATUS_NAMES}.get(status, status)
        e.args = (f"{fn}: {name} ({lib.gn_ops_status_string(status).decode()})",)
        raise e


def _norm_code(norm_type):
    try:
        return _NORM[norm_type]
    except (KeyError, TypeError):
        raise ValueError(f"unsupported norm type {norm_type!r} (2 or inf)") from None


def gn_rms_forward(x, weight, eps=1e-6, *, residual=None, out_dtype=None, need_rstd=True, out=None, h=None,
                   rstd=None):
    """Returns (y, h, rstd): h = x + residual, rounded once to residual's dtype (x itself
    without a residual); rstd = 1 / sqrt(mean(h^2) + eps) over each row, fp32; y = h * rstd *
    weight, computed in fp32 and rounded once to out_dtype (x.dtype or float32; out's by default,
    or x's).

    residual: x's dtype or float32. weight: x's dtype or float32, H elements in any shape, None for
    ones. h=residual updates the residual stream in place, out=x overwrites a contiguous x. rstd,
    which the backward needs, is None with need_rstd=False."""
    y, h, rstd, status = _gnbind.rms_forward(x, weight, eps, residual, _out_code(out_dtype), need_rstd, out, h, rstd)
    _check("gn_rms_forward", status)
    return y, h, rstd


def gn_rms_forward_q8(x, weight, eps=1e-6, *, residual=None, q_dtype=None, block=0, need_rstd=False, out=None,
                      scale=None, h=None, rstd=None):
    """Returns (q, scale, h, rstd): gn_rms_forward's y in 8 bits (torch.int8 or
    torch.float8_e4m3fn; out's dtype by default, or int8) with an fp32 scale for each row
    (block=0) or each run of 32, 64 or 128 columns: scale = max|y| / qmax, q = round(y /
    scale), qmax 127 or 448. scale has x's leading sizes and one more dimension, the scales of
    a row. A run that holds a NaN or an infinity has a NaN scale and zeros."""
    try:
        code = -1 if q_dtype is None else _Q[q_dtype]
    except (KeyError, TypeError):
        raise TypeError(f"unsupported 8-bit dtype {q_dtype} (int8 or float8_e4m3fn)") from None
    q, scale, h, rstd, status = _gnbind.rms_forward_q8(x, weight, eps, residual, code, int(block), need_rstd, out,
                                                       scale, h, rstd)
    _check("gn_rms_forward_q8", status)
    return q, scale, h, rstd


def gn_q8_dequantize(q, scale, out_dtype=None, *, block=0, out=None):
    """q * scale in out_dtype (out's by default, or float32): the values that
    gn_rms_forward_q8's output stands for, for a consumer without an 8-bit form."""
    v, status = _gnbind.q8_dequantize(q, scale, _out_code(out_dtype), int(block), out)
    _check("gn_q8_dequantize", status)
    return v


def gn_rms_workspace_bytes(T, H):
    """Bytes of gn_rms_backward's workspace for T rows of H columns."""
    return int(lib.gn_rms_workspace_bytes(T, H))


def gn_rms_backward(dy, h, rstd, weight, *, dh=None, x_dtype=None, need_dx=True, need_dres=None, need_dweight=True,
                    workspace=None, dx=None, dres=None, dweight=None):
    """Returns (dx, dweight, dres), each None where not needed. h and rstd are
    gn_rms_forward's; dh is the gradient that reaches h through the residual stream (None:
    none). The gradients of x and of the residual are one value, written in x_dtype (h.dtype
    by default) as dx and in h's dtype as dres: one tensor where the dtypes agree and no dres is
    given. need_dres defaults to whether they differ or dres is given. dweight has weight's shape
    and dtype (H float32 elements without a weight). A given output that its flag declines is refused."""
    code = _out_code(x_dtype)
    if need_dres is None:
        need_dres = dres is not None or (x_dtype is not None and x_dtype != h.dtype)
    dx, dweight, dres, status = _gnbind.rms_backward(dy, h, rstd, weight, dh, code, need_dx, need_dres, need_dweight,
                                                     workspace, dx, dres, dweight)
    _check("gn_rms_backward", status)
    return dx, dweight, dres


class RmsNormFn(torch.autograd.Function):
    """(y, h) = the row norm with the HIP kernels in both directions; h is the new residual
    stream, and its gradient joins x's in the backward kernel."""

    @staticmethod
    def forward(ctx, x, weight, eps, residual, out_dtype):
        _gnbind.capture_check([x, weight, residual])
        if not _gnbind.even_rows(x):
            x = x.contiguous()
        residual = residual if residual is None else residual.contiguous()
        y, h, rstd = gn_rms_forward(x, weight, eps, residual=residual, out_dtype=out_dtype)
        ctx.save_for_backward(h, rstd, weight)
        ctx.set_materialize_grads(False)
        ctx.x_dtype, ctx.has_residual = x.dtype, residual is not None
        return (y, h) if ctx.has_residual else y

    @staticmethod
    @once_differentiable
    def backward(ctx, dy, dh=None):
        if dy is None and dh is None:
            return None, None, None, None, None
        h, rstd, weight = ctx.saved_tensors
        need = ctx.needs_input_grad
        if dy is None:  # the stream alone: the norm has no part, also where a row is not finite
            return (dh.to(ctx.x_dtype) if need[0] else None, torch.zeros_like(weight) if need[1] else None, None,
                    dh if need[3] else None, None)
        dx, dweight, dres = gn_rms_backward(
            dy.contiguous(), h, rstd, weight, dh=None if dh is None else dh.contiguous(), x_dtype=ctx.x_dtype, need_dx=need[0],
            need_dres=ctx.has_residual and need[3], need_dweight=weight is not None and need[1])
        return dx, dweight, None, dres, None


def rms_norm(x, weight=None, eps=1e-6, residual=None, out_dtype=None):
    """Root-mean-square norm over the last dimension, differentiable. Returns y, or with a
    residual (y, h), where h = x + residual is the new residual stream and y is its norm."""
    return RmsNormFn.apply(x, weight, eps, residual, out_dtype)


def gn_grad_workspace_bytes(grads):
    """Bytes of the workspace of gn_grad_norm and gn_grad_clip for these tensors' sizes."""
    return _gnbind.grad_workspace_bytes(list(grads))


def gn_grad_norm(grads, norm_type=2.0, *, norm=None, workspace=None):
    """The norm (2 or inf) of all elements of the tensors together, an fp32 scalar on their
    device. Squares are summed in fp64 in a fixed order. float32, bfloat16 and float16 tensors
    may be mixed; each is dense in any order of dimensions."""
    v, status = _gnbind.grads(list(grads), None, False, 0.0, _norm_code(norm_type), norm, workspace)
    _check("gn_grad_norm", status)
    return v


def gn_grad_clip(grads, max_norm, norm_type=2.0, *, out=None, norm=None, workspace=None):
    """Scales the tensors by min(1, max_norm / (norm + 1e-6)), in place or into `out` (tensors
    of the same shapes and element orders, in the gradients' dtype or float32), and returns the norm
    from before. The factor is decided on the device; an infinite max_norm clips nothing."""
    v, status = _gnbind.grads(list(grads), None if out is None else list(out), True, float(max_norm),
                              _norm_code(norm_type), norm, workspace)
    _check("gn_grad_clip", status)
    return v


def clip_gradients(parameters, max_norm, norm_type=2.0):
    """Clips the gradients of the parameters (a tensor or an iterable; those without a
    gradient are passed over) in place by their norm together, which is returned. A parameter
    listed twice counts once. The gradients are dense, on one device (gradients on several are
    refused), and none overlaps another."""
    parameters = [parameters] if isinstance(parameters, torch.Tensor) else list(parameters)
    grads = list({id(p): p.grad for p in parameters if p.grad is not None}.values())
    if not grads:
        return torch.tensor(0.0)
    return gn_grad_clip(grads, max_norm, norm_type)
