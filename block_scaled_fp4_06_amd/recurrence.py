"""A gated linear recurrence over time.

Per batch row and channel:

  a_t = floor + (1 - floor) sigmoid(g_t),   h_t = a_t h_{t-1} + (1 - a_t) u_t,   y_t = h_t

g and u are (batch, time, chan) with unit channel stride and any other strides (the two halves
of one projection, for example), both bf16 or both float32; y and the gradients take their
type.  floor (chan,) and the states (batch, chan) are float32; the state is carried in
float32 throughout.  reset (batch, time, bool or uint8) marks the first step of each document
of a packed row: there h_t = u_t, and nothing that came before has any influence.  A gate of
+inf leaves a step out (a = 1), one of -inf gives a = floor.

``gated_scan_forward`` with time 1 is a decoder's step.  ``autograd_gated_scan()`` wraps the
calls for torch.autograd.
"""
from __future__ import annotations

from dataclasses import dataclass
from typing import Optional

from . import nvfp4 as N
from .launch import check, dtype_code, new_like, ptr, run_on


@dataclass
class GatedScanGrads:
    dg: "object"
    du: "object"
    dh0: "object"
    dfloor: Optional["object"]


def _sequence(name, t, like):
    if t.shape != like.shape:
        raise ValueError("%s has shape %s, expected %s" % (name, tuple(t.shape),
                                                           tuple(like.shape)))
    if t.dtype is not like.dtype:
        raise ValueError("%s has dtype %s, expected %s" % (name, t.dtype, like.dtype))
    if t.device != like.device:
        raise ValueError("%s is on %s, expected %s" % (name, t.device, like.device))
    batch, time, chan = t.shape
    if not t.is_contiguous() and t.numel() and (
            (chan > 1 and t.stride(2) != 1) or (time > 1 and t.stride(1) < chan)):
        raise ValueError("%s must have unit channel stride and time steps apart" % name)


def _state(name, t, shape, like):
    import torch
    if t is None:
        return
    N._check_buffer(name, t, shape, (torch.float32,), like.device, False)


def _check_inputs(g, u, floor, h0, reset):
    import torch
    if g.dim() != 3:
        raise ValueError("g must be (batch, time, chan), not %d-D" % g.dim())
    dtype_code("g", g)
    _sequence("g", g, g)
    _sequence("u", u, g)
    batch, time, chan = g.shape
    _state("floor", floor, (chan,), g)
    _state("h0", h0, (batch, chan), g)
    if reset is not None:
        N._check_buffer("reset", reset, (batch, time), (torch.bool, torch.uint8), g.device, False)


def _strides(t):
    batch, time, _ = t.shape
    b, t, _ = t.stride()
    return (b if batch > 1 else 0), (t if time > 1 else 0)


def _args(g, u, floor, h0, reset, y, h_last):
    batch, time, chan = g.shape
    return N.ScanArgs(batch, time, chan, dtype_code("g", g), 0, ptr(g), *_strides(g), ptr(u),
                      *_strides(u), ptr(floor), ptr(h0), ptr(reset), ptr(y), *_strides(y),
                      ptr(h_last))


def gated_scan_forward(g, u, floor=None, h0=None, reset=None, h_last=None, stream=None):
    """(y, h_last): every step's state in the type of g, and the last one in float32 (into
    h_last where given; h0 itself for a state kept in place)."""
    import torch
    _check_inputs(g, u, floor, h0, reset)
    batch, time, chan = g.shape
    _state("h_last", h_last, (batch, chan), g)
    dev, given = g.device, h_last

    def call(handle):
        y = new_like(g)
        last = given if given is not None else (
            torch.empty((batch, chan), dtype=torch.float32, device=dev))
        need = N.nvfp4_gated_scan_workspace_bytes(batch, time, chan, 0)
        ws = torch.empty(need, dtype=torch.uint8, device=dev) if need else None
        check(N.nvfp4_gated_scan_forward(_args(g, u, floor, h0, reset, y, last), ptr(ws), need,
                                         handle), "nvfp4_gated_scan_forward")
        return y, last
    y, h_last = run_on(stream, dev, (g, u, floor, h0, reset, given), call)
    if given is not None:
        torch.autograd.graph.increment_version(given)
    return y, h_last


def gated_scan_backward(dy, g, u, y, floor=None, h0=None, reset=None, dh_last=None,
                        stream=None, out=None) -> GatedScanGrads:
    """The gradients of gated_scan_forward from those of y (dy) and of h_last (dh_last, None:
    zero); y as the forward call returned it.  out: (dg, du) to write into, laid out as g and
    u may be (the two halves of one projection's gradient, for example); neither may share
    memory with an input."""
    import torch
    _check_inputs(g, u, floor, h0, reset)
    _sequence("dy", dy, g)
    _sequence("y", y, g)
    batch, time, chan = g.shape
    _state("dh_last", dh_last, (batch, chan), g)
    if out is not None:
        _sequence("out[0]", out[0], g)
        _sequence("out[1]", out[1], g)
    dev = g.device

    def call(handle):
        dg, du = (new_like(g), new_like(g)) if out is None else out
        dh0 = torch.empty((batch, chan), dtype=torch.float32, device=dev)
        dfloor = None if floor is None else torch.empty_like(floor)
        need = N.nvfp4_gated_scan_workspace_bytes(batch, time, chan, 1)
        ws = torch.empty(need, dtype=torch.uint8, device=dev)
        grads = N.ScanGradArgs(ptr(dy), *_strides(dy), ptr(dh_last), ptr(dg), *_strides(dg),
                               ptr(du), *_strides(du), ptr(dh0), ptr(dfloor))
        check(N.nvfp4_gated_scan_backward(_args(g, u, floor, h0, reset, y, None), grads, ptr(ws),
                                          need, handle), "nvfp4_gated_scan_backward")
        return GatedScanGrads(dg, du, dh0, dfloor)
    return run_on(stream, dev, (dy, g, u, y, floor, h0, reset, dh_last, *(out or ())), call)


_AUTOGRAD = {}


def autograd_gated_scan():
    """A torch.autograd.Function: (y, h_last) = apply(g, u, floor, h0, reset); floor, h0 and
    reset may be None."""
    if "scan" in _AUTOGRAD:
        return _AUTOGRAD["scan"]
    import torch

    class GatedScanFn(torch.autograd.Function):
        @staticmethod
        def forward(fctx, g, u, floor, h0, reset):
            y, h_last = gated_scan_forward(g, u, floor, h0, reset)
            fctx.save_for_backward(g, u, y, floor, h0, reset)
            return y, h_last

        @staticmethod
        def backward(fctx, dy, dh_last):
            g, u, y, floor, h0, reset = fctx.saved_tensors
            d = gated_scan_backward(dy.contiguous(), g, u, y, floor, h0, reset,
                                    dh_last.contiguous())
            return d.dg, d.du, d.dfloor, None if h0 is None else d.dh0, None

    _AUTOGRAD["scan"] = GatedScanFn
    return GatedScanFn
