"""A recurrent residual block on NVFP4 linear layers: forward, backward and one decoding step.

  (g | u) = h W_in              NVFP4 linear (linear.py), h the block's normed input
  y       = scan(g, u)          gated linear recurrence over time (recurrence.py)
  z       = y W_out             NVFP4 linear
  x_out   = skip x + branch gate norm(z),   h_next = norm(x_out)        (norm.py)

h_next is the next block's h.  x and h are (batch * time, dim), time steps of one sequence
consecutive; batch * time and dim are multiples of 16 (the quantizer's unit).  This module
only sequences the library's calls.
"""
from __future__ import annotations

from dataclasses import dataclass, fields
from typing import Optional

from . import linear as L
from . import norm
from . import recurrence as R
from .launch import run_on, tensors_in


@dataclass
class BlockParams:
    """Parameters of one block (or their gradients)."""
    w_in: "object"          # (dim, 2 dim) bf16: gates, then inputs of the recurrence
    w_out: "object"         # (dim, dim) bf16
    floor: "object"         # (dim,) float32, the decay's floor, in [0, 1)
    post_weight: "object"   # (dim,) float32, norm of the block's output
    gate: "object"          # (1, dim) float32
    next_weight: "object"   # (dim,) float32, norm before the next block

    def tensors(self):
        return [getattr(self, f.name) for f in fields(self)]


@dataclass
class BlockContext:
    """What the backward pass keeps from the forward pass."""
    lin_in: L.LinearContext
    lin_out: L.LinearContext
    gu: "object"
    y: "object"
    floor: "object"
    h0: Optional["object"]
    reset: Optional["object"]
    norm: norm.ResidualNormContext


def new_block(dim, device, seed=0, branch_init=0.5) -> BlockParams:
    """Random weights of a block (normal, variance 1 / fan-in), unit norms, decay floors
    spread over [0, 0.9]."""
    import torch
    gen = torch.Generator(device="cpu").manual_seed(seed)
    std = dim ** -0.5

    def weight(rows, cols):
        return (torch.randn(rows, cols, generator=gen) * std).to(torch.bfloat16).to(device)
    return BlockParams(weight(dim, 2 * dim), weight(dim, dim),
                       torch.linspace(0.0, 0.9, dim).to(device), torch.ones(dim, device=device),
                       torch.full((1, dim), branch_init, device=device),
                       torch.ones(dim, device=device))


def block_forward(x, h, p: BlockParams, batch, time, h0=None, reset=None, sr_seed=0,
                  skip_scale=1.0, branch_scale=1.0, eps=1e-6, stream=None):
    """(x_out, h_next, state, ctx); state (batch, dim) float32 is the recurrence's after the
    last step, h0 the one before the first."""
    def call(_):   # (with `stream` current: what lies between the calls belongs to it too)
        dim = x.shape[1]
        gu, lin_in = L.linear_forward(h, p.w_in, sr_seed=sr_seed)
        gu = gu.view(batch, time, 2 * dim)
        y, state = R.gated_scan_forward(gu[:, :, :dim], gu[:, :, dim:], p.floor, h0, reset)
        z, lin_out = L.linear_forward(y.view(batch * time, dim), p.w_out, sr_seed=sr_seed + 2)
        x_out, h_next, ctx = norm.residual_norm_forward(x, z, p.post_weight, p.next_weight, p.gate,
                                                        skip_scale, branch_scale, eps)
        return x_out, h_next, state, BlockContext(lin_in, lin_out, gu, y, p.floor, h0, reset, ctx)
    used = () if stream is None else list(tensors_in(x, h, p, h0, reset))
    return run_on(stream, x.device, used, call)


def block_backward(dx_out, dh_next, ctx: BlockContext, dstate=None, stream=None):
    """(dx, dh, dh0, gradients as a BlockParams) from the gradients of block_forward's
    results (dx_out None: zero; dstate None: zero)."""
    import torch

    def call(_):
        batch, time, dim = ctx.y.shape
        d = norm.residual_norm_backward(dx_out, dh_next, ctx.norm)
        dy, dw_out = L.linear_backward(d.dz, ctx.lin_out, dw_dtype=torch.bfloat16)
        dgu = torch.empty_like(ctx.gu)
        g, u = ctx.gu[:, :, :dim], ctx.gu[:, :, dim:]
        s = R.gated_scan_backward(dy.view(batch, time, dim), g, u, ctx.y, ctx.floor, ctx.h0,
                                  ctx.reset, dstate, out=(dgu[:, :, :dim], dgu[:, :, dim:]))
        dh, dw_in = L.linear_backward(dgu.view(batch * time, 2 * dim), ctx.lin_in,
                                      dw_dtype=torch.bfloat16)
        grads = BlockParams(dw_in, dw_out, s.dfloor, d.dpost_weight, d.dgate, d.dnext_weight)
        return d.dx, dh, s.dh0, grads
    used = () if stream is None else list(tensors_in(dx_out, dh_next, ctx, dstate))
    return run_on(stream, ctx.y.device, used, call)
