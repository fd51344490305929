"""The norms before and after a block, its gate and the scaled residual sum.

One call closes a block and opens the next:

  n2    = z / sqrt(mean(z^2) + eps)                                   (per row)
  x_out = skip_scale x + branch_scale gate (n2 (weight_offset + post_weight))
  h     = x_out / sqrt(mean(x_out^2) + eps) (weight_offset + next_weight)

with z the block's output, x the residual stream before it and h the next block's input,
and one call gives all the gradients.  ``norm_forward`` / ``norm_backward`` are the norm of
the stream alone (the first block's input, a model's last norm).

x, z are 2-D (rows, cols) with unit column stride, any row stride, bf16 or float32 (z bf16
where x is); x_out and the gradients of x take x's type, h and dz take z's.  The weights are
1-D, bf16 or float32; gate is (gate_rows, cols) with gate_rows dividing rows, each gate row
shared by rows / gate_rows consecutive rows: (1, cols) is a gate per channel, (batch, cols)
one per sample, (rows, cols) one per token.  Statistics and sums are float32 and the sums
over rows are taken in a fixed order.  ``autograd_residual_norm()`` and ``autograd_norm()``
wrap the calls for torch.autograd.
"""
from __future__ import annotations

from dataclasses import dataclass
from typing import Optional

from . import nvfp4 as N
from .launch import apart, check, dtype_code, new_like, ptr, run_on

MAX_COLS = 32768


@dataclass
class ResidualNormContext:
    """What the backward pass reads: stored by the forward call."""
    x_out: "object"
    z: Optional["object"]
    post_weight: Optional["object"]
    next_weight: Optional["object"]
    gate: Optional["object"]
    rstd: Optional["object"]
    rstd_post: Optional["object"]
    skip_scale: float = 1.0
    branch_scale: float = 1.0
    weight_offset: float = 0.0


@dataclass
class ResidualNormGrads:
    dx: "object"
    dz: Optional["object"]
    dpost_weight: Optional["object"]
    dnext_weight: Optional["object"]
    dgate: Optional["object"]


def _matrix(name, t, shape, device, dtype=None):
    """t is a (rows, cols) tensor of `shape` on `device` with rows laid out apart."""
    if t.shape != shape:
        raise ValueError("%s has shape %s, expected %s" % (name, tuple(t.shape), tuple(shape)))
    if dtype is None:
        dtype_code(name, t)
    elif t.dtype is not dtype:
        raise ValueError("%s has dtype %s, expected %s" % (name, t.dtype, dtype))
    if t.device != device:
        raise ValueError("%s is on %s, expected %s" % (name, t.device, device))
    rows, cols = shape
    if not t.is_contiguous() and ((cols > 1 and rows and t.stride(1) != 1) or
                                  (rows > 1 and cols and t.stride(0) < cols)):
        raise ValueError("%s must be row-major with unit column stride" % name)


def _vector(name, t, n, device, dtype=None):
    if t.dim() != 1 or t.shape[0] != n:
        raise ValueError("%s has shape %s, expected (%d,)" % (name, tuple(t.shape), n))
    if dtype is None:
        dtype_code(name, t)
    elif t.dtype is not dtype:
        raise ValueError("%s has dtype %s, expected %s" % (name, t.dtype, dtype))
    if t.device != device:
        raise ValueError("%s is on %s, expected %s" % (name, t.device, device))
    if not t.is_contiguous():
        raise ValueError("%s must be contiguous" % name)


def _check_operands(x, z, post_weight, next_weight, gate):
    if x.dim() != 2:
        raise ValueError("x must be 2-D, not %d-D" % x.dim())
    shape, device = x.shape, x.device
    rows, cols = shape
    if cols > MAX_COLS:
        raise ValueError("x has %d columns, at most %d are supported" % (cols, MAX_COLS))
    _matrix("x", x, shape, device)
    if z is None:
        if post_weight is not None or gate is not None:
            raise ValueError("post_weight and gate need a branch z")
        if next_weight is None:
            raise ValueError("next_weight is missing")
    else:
        _matrix("z", z, shape, device)
        if z.dtype is not x.dtype and dtype_code("x", x) == 0:
            raise ValueError("z has dtype %s, expected %s" % (z.dtype, x.dtype))
        if post_weight is None:
            raise ValueError("post_weight is missing")
        _vector("post_weight", post_weight, cols, device)
    if next_weight is not None:
        _vector("next_weight", next_weight, cols, device,
                None if post_weight is None else post_weight.dtype)
    if gate is not None:
        if gate.dim() != 2:
            raise ValueError("gate must be 2-D, not %d-D" % gate.dim())
        g = gate.shape[0]
        if g < 1 or rows % g or (rows and g > rows):
            raise ValueError("gate has %d rows, which must divide the %d rows of x" % (g, rows))
        _matrix("gate", gate, (g, cols), device)


def _params(x, h_type_of, weight, gate, eps, offset, skip, branch):
    rows, cols = x.shape
    return N.NormParams(rows, cols, 1 if gate is None else gate.shape[0], dtype_code("x", x),
                        dtype_code("z", h_type_of), dtype_code("weight", weight),
                        0 if gate is None else dtype_code("gate", gate), eps, offset, skip, branch)


def _ld(t):
    return t.stride(0) if t is not None else 0


def residual_norm_forward(x, z, post_weight, next_weight=None, gate=None, skip_scale=1.0,
                          branch_scale=1.0, eps=1e-6, weight_offset=0.0, out=None, stream=None):
    """(x_out, h, ctx): the end of one block and the beginning of the next.

    next_weight None: only the sum is formed and h is None.  out: where x_out goes (shape and
    type of x; x itself for an update in place, and no memory of another input)."""
    import torch
    if z is None:
        raise ValueError("z is missing (norm_forward is the norm without a branch)")
    _check_operands(x, z, post_weight, next_weight, gate)
    if out is not None:
        _matrix("out", out, x.shape, x.device, x.dtype)
        in_place = out is x or (out.data_ptr() == x.data_ptr() and out.stride() == x.stride())
        for name, t in (("x", None if in_place else x), ("z", z), ("post_weight", post_weight),
                        ("next_weight", next_weight), ("gate", gate)):
            if not apart(out, t):
                raise ValueError("out shares memory with %s" % name)
    ctx = ResidualNormContext(out, z, post_weight, next_weight, gate, None, None, skip_scale,
                              branch_scale, weight_offset)

    def call(handle):
        dev, f32 = x.device, torch.float32
        x_out = ctx.x_out = new_like(x) if out is None else out
        ctx.rstd_post = torch.empty(x.shape[0], dtype=f32, device=dev)
        h = None
        if next_weight is not None:
            h = new_like(z)
            ctx.rstd = torch.empty(x.shape[0], dtype=f32, device=dev)
        prm = _params(x, z, post_weight, gate, eps, weight_offset, skip_scale, branch_scale)
        args = N.NormForwardArgs(ptr(x), _ld(x), ptr(z), _ld(z), ptr(post_weight), ptr(gate),
                                 _ld(gate), ptr(next_weight), ptr(x_out), _ld(x_out), ptr(h),
                                 _ld(h), ptr(ctx.rstd), ptr(ctx.rstd_post))
        check(N.nvfp4_residual_norm_forward(prm, args, handle), "nvfp4_residual_norm_forward")
        return h
    h = run_on(stream, x.device, (x, z, post_weight, next_weight, gate, out), call)
    if out is not None:
        torch.autograd.graph.increment_version(out)
    return ctx.x_out, h, ctx


def norm_forward(x, weight, eps=1e-6, weight_offset=0.0, out_dtype=None, stream=None):
    """(h, ctx): h = x / sqrt(mean(x^2) + eps) (weight_offset + weight), of out_dtype (default
    x's; bf16 where x is)."""
    import torch
    _check_operands(x, None, None, weight, None)
    out_dtype = out_dtype or x.dtype
    if out_dtype not in (torch.bfloat16, torch.float32) or (
            x.dtype == torch.bfloat16 and out_dtype != x.dtype):
        raise ValueError("out_dtype %s does not go with x of %s" % (out_dtype, x.dtype))
    def call(handle):
        h = torch.empty(x.shape, dtype=out_dtype, device=x.device)
        rstd = torch.empty(x.shape[0], dtype=torch.float32, device=x.device)
        prm = _params(x, h, weight, None, eps, weight_offset, 1.0, 1.0)
        args = N.NormForwardArgs(x=ptr(x), ld_x=_ld(x), next_weight=ptr(weight), h=ptr(h),
                                 ld_h=_ld(h), rstd=ptr(rstd))
        check(N.nvfp4_residual_norm_forward(prm, args, handle), "nvfp4_residual_norm_forward")
        return h, rstd
    h, rstd = run_on(stream, x.device, (x, weight), call)
    return h, ResidualNormContext(x, None, None, weight, None, rstd, None, 1.0, 1.0, weight_offset)


def residual_norm_backward(dx_out, dh, ctx: ResidualNormContext, stream=None) -> ResidualNormGrads:
    """The gradients of residual_norm_forward (or norm_forward) from those of its outputs:
    dx_out None where only h was used, dh None where next_weight was None."""
    import torch
    x, z, gate = ctx.x_out, ctx.z, ctx.gate
    _check_operands(x, z, ctx.post_weight, ctx.next_weight, gate)
    rows, cols = x.shape
    dev, f32 = x.device, torch.float32
    if dx_out is not None:
        _matrix("dx_out", dx_out, x.shape, dev, x.dtype)
    if (dh is None) != (ctx.next_weight is None):
        raise ValueError("dh must be given exactly when the forward call had next_weight")
    if dh is not None:
        _matrix("dh", dh, x.shape, dev, None if z is None else z.dtype)
        _vector("rstd", ctx.rstd, rows, dev, f32)
    if z is not None:
        _vector("rstd_post", ctx.rstd_post, rows, dev, f32)

    def call(handle):
        d = ResidualNormGrads(new_like(x), new_like(z), new_like(ctx.post_weight),
                              new_like(ctx.next_weight), new_like(gate))
        prm = _params(x, dh if z is None else z,
                      ctx.next_weight if ctx.post_weight is None else ctx.post_weight, gate, 0.0,
                      ctx.weight_offset, ctx.skip_scale, ctx.branch_scale)
        need = N.nvfp4_residual_norm_workspace_bytes(prm)
        ws = torch.empty(need, dtype=torch.uint8, device=dev)
        args = N.NormBackwardArgs(ptr(x), _ld(x), ptr(z), _ld(z), ptr(ctx.post_weight), ptr(gate),
                                  _ld(gate), ptr(ctx.next_weight), ptr(ctx.rstd),
                                  ptr(ctx.rstd_post), ptr(dx_out), _ld(dx_out), ptr(dh), _ld(dh),
                                  ptr(d.dx), _ld(d.dx), ptr(d.dz), _ld(d.dz), ptr(d.dpost_weight),
                                  ptr(d.dnext_weight), ptr(d.dgate), _ld(d.dgate))
        check(N.nvfp4_residual_norm_backward(prm, args, ptr(ws), need, handle),
              "nvfp4_residual_norm_backward")
        return d
    return run_on(stream, dev, (x, z, ctx.post_weight, ctx.next_weight, gate, ctx.rstd,
                                ctx.rstd_post, dx_out, dh), call)


def norm_backward(dh, ctx: ResidualNormContext, dresidual=None, stream=None):
    """(dx, dweight) of norm_forward; dresidual, the gradient that x receives from elsewhere,
    is added to dx."""
    if ctx.z is not None:
        raise ValueError("the context is residual_norm_forward's")
    d = residual_norm_backward(dresidual, dh, ctx, stream=stream)
    return d.dx, d.dnext_weight


_AUTOGRAD = {}


def _rows_apart(t):
    """A gradient as the calls take it: autograd may hand over expanded or transposed ones."""
    return t if t is None or (t.dim() == 2 and t.is_contiguous()) else t.contiguous()


def autograd_residual_norm():
    """A torch.autograd.Function: (x_out, h) = apply(x, z, post_weight, next_weight, gate,
    skip_scale, branch_scale, eps, weight_offset); next_weight and gate may be None (h is then
    None)."""
    if "residual" in _AUTOGRAD:
        return _AUTOGRAD["residual"]
    import torch

    class ResidualNormFn(torch.autograd.Function):
        @staticmethod
        def forward(fctx, x, z, post_weight, next_weight, gate, skip_scale, branch_scale, eps,
                    weight_offset):
            x_out, h, c = residual_norm_forward(x, z, post_weight, next_weight, gate, skip_scale,
                                                branch_scale, eps, weight_offset)
            fctx.save_for_backward(c.x_out, z, post_weight, next_weight, gate, c.rstd, c.rstd_post)
            fctx.scales = (skip_scale, branch_scale, weight_offset)
            return x_out, h

        @staticmethod
        @torch.autograd.function.once_differentiable
        def backward(fctx, dx_out, dh):
            d = residual_norm_backward(_rows_apart(dx_out), _rows_apart(dh),
                                       ResidualNormContext(*fctx.saved_tensors, *fctx.scales))
            return d.dx, d.dz, d.dpost_weight, d.dnext_weight, d.dgate, None, None, None, None

    _AUTOGRAD["residual"] = ResidualNormFn
    return ResidualNormFn


def autograd_norm():
    """A torch.autograd.Function: h = apply(x, weight, eps, weight_offset)."""
    if "norm" in _AUTOGRAD:
        return _AUTOGRAD["norm"]
    import torch

    class NormFn(torch.autograd.Function):
        @staticmethod
        def forward(fctx, x, weight, eps, weight_offset):
            h, c = norm_forward(x, weight, eps, weight_offset)
            fctx.save_for_backward(x, weight, c.rstd)
            fctx.weight_offset = weight_offset
            return h

        @staticmethod
        @torch.autograd.function.once_differentiable
        def backward(fctx, dh):
            x, weight, rstd = fctx.saved_tensors
            ctx = ResidualNormContext(x, None, None, weight, None, rstd, None, 1.0, 1.0,
                                      fctx.weight_offset)
            dx, dweight = norm_backward(_rows_apart(dh), ctx)
            return dx, dweight, None, None

    _AUTOGRAD["norm"] = NormFn
    return NormFn
