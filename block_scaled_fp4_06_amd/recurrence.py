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
from .launch import apart, check, dtype_code, new_like, ptr, run_on


@dataclass
class GatedScanGrads:
    dg: "object"
    du: "object"
    dh0: "object"
    dfloor: Optional["object"]


def _sequence(name, t, shape, dtype, device):
    if t.shape != shape:
        raise ValueError("%s has shape %s, expected %s" % (name, tuple(t.shape), tuple(shape)))
    if t.dtype is not dtype:
        raise ValueError("%s has dtype %s, expected %s" % (name, t.dtype, dtype))
    if t.device != device:
        raise ValueError("%s is on %s, expected %s" % (name, t.device, device))
    _steps(name, t, shape)


def _steps(name, t, shape):
    if t.is_contiguous() or not t.numel():
        return
    _, time, chan = shape
    if (chan > 1 and t.stride(2) != 1) or (time > 1 and t.stride(1) < chan):
        raise ValueError("%s must have unit channel stride and time steps apart" % name)


def _output(name, t, chan):
    """No two steps of t share memory (an expanded tensor's would)."""
    (s0, n0), (s1, n1) = sorted(zip(_strides(t), t.shape))   # (0 for a single row or step)
    if t.numel() and ((n0 > 1 and s0 < chan) or (n1 > 1 and s1 < (n0 - 1) * s0 + chan)):
        raise ValueError("%s must have rows and time steps apart" % name)


def _plain(name, t, shape, dtypes, device):
    if t is not None and (t.shape != shape or t.dtype not in dtypes or t.device != device or
                          not t.is_contiguous()):
        N._check_buffer(name, t, shape, dtypes, device, False)   # (says what is wrong)


def _check_inputs(g, u, floor, h0, reset):
    """The shape, type and device that the other tensors share with g."""
    import torch
    if g.dim() != 3:
        raise ValueError("g must be (batch, time, chan), not %d-D" % g.dim())
    dtype_code("g", g)
    shape, dtype, device = g.shape, g.dtype, g.device
    _steps("g", g, shape)
    _sequence("u", u, shape, dtype, device)
    batch, time, chan = shape
    f32 = (torch.float32,)
    _plain("floor", floor, (chan,), f32, device)
    _plain("h0", h0, (batch, chan), f32, device)
    _plain("reset", reset, (batch, time), (torch.bool, torch.uint8), device)
    return shape, dtype, device


def _strides(t):
    batch, time, chan = t.shape
    if t.is_contiguous():
        b, t = time * chan, chan
    else:
        b, t, _ = t.stride()
    return (b if batch > 1 else 0), (t if time > 1 else 0)


def _args(g, u, floor, h0, reset, y, h_last):
    batch, time, chan = g.shape
    return N.ScanArgs(batch, time, chan, dtype_code("g", g), 0, ptr(g), *_strides(g), ptr(u),
                      *_strides(u), ptr(floor), ptr(h0), ptr(reset), ptr(y), *_strides(y),
                      ptr(h_last))


def gated_scan_forward(g, u, floor=None, h0=None, reset=None, h_last=None, stream=None):
    """(y, h_last): every step's state in the type of g, and the last one in float32 (into
    h_last where given: h0 itself for a state kept in place, or memory of no input)."""
    import torch
    (batch, time, chan), _, dev = _check_inputs(g, u, floor, h0, reset)
    _plain("h_last", h_last, (batch, chan), (torch.float32,), dev)
    if h_last is not None and h_last is not h0:
        for name, t in (("h0", None if ptr(h0) == ptr(h_last) else h0), ("g", g), ("u", u),
                        ("floor", floor), ("reset", reset)):
            if not apart(h_last, t):
                raise ValueError("h_last shares memory with %s" % name)
    given = h_last

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
    memory with the other or with an input."""
    import torch
    shape, dtype, dev = _check_inputs(g, u, floor, h0, reset)
    _sequence("dy", dy, shape, dtype, dev)
    _sequence("y", y, shape, dtype, dev)
    batch, time, chan = shape
    _plain("dh_last", dh_last, (batch, chan), (torch.float32,), dev)
    if out is not None:
        _sequence("out[0]", out[0], shape, dtype, dev)
        _sequence("out[1]", out[1], shape, dtype, dev)
        _output("out[0]", out[0], chan)
        _output("out[1]", out[1], chan)
        if not apart(*out):
            raise ValueError("out[0] and out[1] share memory")
        for name, t in zip(("dy", "g", "u", "y", "floor", "h0", "reset", "dh_last"),
                           (dy, g, u, y, floor, h0, reset, dh_last)):
            if not apart(out[0], t) or not apart(out[1], t):
                raise ValueError("out shares memory with %s" % name)

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
    grads = run_on(stream, dev, (dy, g, u, y, floor, h0, reset, dh_last, *(out or ())), call)
    if out is not None:
        torch.autograd.graph.increment_version(out)
    return grads


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
        @torch.autograd.function.once_differentiable
        def backward(fctx, dy, dh_last):
            g, u, y, floor, h0, reset = fctx.saved_tensors
            d = gated_scan_backward(dy.contiguous(), g, u, y, floor, h0, reset,
                                    dh_last.contiguous())
            return d.dg, d.du, d.dfloor, None if h0 is None else d.dh0, None

    _AUTOGRAD["scan"] = GatedScanFn
    return GatedScanFn
