"""AdamW over many tensors in one launch, moments in 32 or in 8 bits.

  m = beta1 m + (1 - beta1) g;   v = beta2 v + (1 - beta2) g^2
  w = w (1 - lr weight_decay) - lr / (1 - beta1^t) m / (sqrt(v / (1 - beta2^t)) + eps)

Parameters are bf16 or float32, of any size.  A bf16 parameter may have a float32 master
copy, which then is what the update works on; without one it is rounded to nearest, or
stochastically (``stochastic_rounding=True``: small updates survive on average).

The moments of all parameters live in flat buffers (``AdamWState``), each parameter's share
beginning at a multiple of 256 elements.  8-bit moments hold, per block of 256 elements of a
parameter, one float32 scale (a power of two) and a byte per element: E4M3 codes for the first
moment (nearest, so beta1 is at most 17/18: above, a moment whose gradient has vanished would
stay while the second one decays, and its parameter run away), and for the second the root of v as an unsigned float of 4 exponent and 4
mantissa bits, rounded stochastically (rounding to nearest would freeze it: beta2 near 1 moves v
by less than half a code per step).  The draws come from Philox4x32-10 keyed on (seed, step, parameter, element),
so a step's result is a function of its inputs alone.

The step number and lr are arguments of the launch: a captured HIP graph of a step would
repeat that step's values.
"""
from __future__ import annotations

from dataclasses import dataclass
from struct import Struct
from typing import Optional

from . import nvfp4 as N
from .launch import check, dtype_code, ptr, run_on

BLOCK = 256   # elements of one block of 8-bit moments (NVFP4_ADAMW_BLOCK)
MAX_BETA1_8 = 17.0 / 18.0   # of 8-bit moments (NVFP4_ADAMW_MAX_BETA1_8)


@dataclass
class AdamWState:
    """Flat state of a list of parameters: parameter i's share begins at offsets(params)[i].

    bits 32: exp_avg, exp_avg_sq float32.  bits 8: uint8 codes, and float32 scales per 256
    elements.  master: float32 copies of the parameters, or None."""
    bits: int
    exp_avg: "object"
    exp_avg_sq: "object"
    exp_avg_scale: Optional["object"] = None
    exp_avg_sq_scale: Optional["object"] = None
    master: Optional["object"] = None
    step: int = 0


def offsets(params):
    """Where each parameter's share of the flat state begins, and the state's length."""
    at, end = [], 0
    for p in params:
        at.append(end)
        end += -(-p.numel() // BLOCK) * BLOCK
    return at, end


def new_state(params, bits=32, master=False) -> AdamWState:
    """Zero moments for `params`, and with master=True float32 copies of their values."""
    import torch
    if bits not in (32, 8):
        raise ValueError("bits must be 32 or 8, not %r" % (bits,))
    params = list(params)
    if not params:
        raise ValueError("no parameters")
    dev = params[0].device
    at, end = offsets(params)
    copies = None
    if master:
        copies = torch.zeros(end, dtype=torch.float32, device=dev)
        for a, p in zip(at, params):
            copies[a:a + p.numel()].copy_(p.detach().reshape(-1))
    if bits == 32:
        return AdamWState(32, torch.zeros(end, dtype=torch.float32, device=dev),
                          torch.zeros(end, dtype=torch.float32, device=dev), master=copies)
    return AdamWState(8, torch.zeros(end, dtype=torch.uint8, device=dev),
                      torch.zeros(end, dtype=torch.uint8, device=dev),
                      torch.zeros(end // BLOCK, dtype=torch.float32, device=dev),
                      torch.zeros(end // BLOCK, dtype=torch.float32, device=dev), copies)


class AdamW:
    """The optimizer of a fixed list of parameters (contiguous tensors on one GPU, none of
    which shares memory with another: a tied weight is listed once).

    weight_decay: one number, or one per parameter.  state: an AdamWState to go on with;
    by default new_state(params, bits, master).  Tensors in `state` are used, not copied."""

    def __init__(self, params, lr=1e-3, betas=(0.9, 0.999), eps=1e-8, weight_decay=0.0, bits=32,
                 master=False, state: Optional[AdamWState] = None, stochastic_rounding=False,
                 seed=0):
        self.params = list(params)
        if not self.params:
            raise ValueError("no parameters")
        self.device = self.params[0].device
        self._shapes = [p.shape for p in self.params]
        self._check_params()
        if not 0.0 <= betas[0] < 1.0 or not 0.0 <= betas[1] < 1.0:
            raise ValueError("betas must lie in [0, 1), not %r" % (betas,))
        if not eps >= 0.0:
            raise ValueError("eps must not be negative")
        self.lr, self.betas, self.eps = lr, tuple(betas), eps
        self.weight_decay = weight_decay
        self.stochastic_rounding, self.seed = bool(stochastic_rounding), int(seed)
        self.state = state if state is not None else new_state(self.params, bits, master)
        self._check_state()
        if self.state.bits == 8 and self.betas[0] > MAX_BETA1_8:
            raise ValueError("betas[0] is %r, at most 17/18 is supported with 8-bit moments" %
                             (self.betas[0],))
        self._pack = Struct("=%dQ" % len(self.params)).pack
        self._table = None

    @property
    def weight_decay(self):
        """One number per parameter; an assignment also takes one for all.  What a step finds
        here is what it applies, as with lr, betas and eps."""
        return self._weight_decay

    @weight_decay.setter
    def weight_decay(self, value):
        decay = value if isinstance(value, (list, tuple)) else [value] * len(self.params)
        if len(decay) != len(self.params):
            raise ValueError("%d weight_decay values for %d parameters" % (len(decay),
                                                                           len(self.params)))
        self._weight_decay = [float(d) for d in decay]

    def _check_params(self):
        for i, (p, shape) in enumerate(zip(self.params, self._shapes)):
            dtype_code("params[%d]" % i, p)
            if p.device != self.device:
                raise ValueError("params[%d] is on %s, expected %s" % (i, p.device, self.device))
            if p.shape != shape:
                raise ValueError("params[%d] has shape %s, expected %s" % (i, tuple(p.shape),
                                                                           tuple(shape)))
            if not p.is_contiguous():
                raise ValueError("params[%d] must be contiguous" % i)
        spans = sorted((p.data_ptr(), p.data_ptr() + p.numel() * p.element_size(), i)
                       for i, p in enumerate(self.params) if p.numel())
        for (_, end, i), (begin, _, j) in zip(spans, spans[1:]):
            if begin < end:   # (two workgroups would update the same elements)
                raise ValueError("params[%d] and params[%d] share memory" % (min(i, j), max(i, j)))

    def _check_state(self):
        import torch
        s, (_, end) = self.state, offsets(self.params)
        if s.bits not in (32, 8):
            raise ValueError("state.bits must be 32 or 8, not %r" % (s.bits,))
        kind = torch.float32 if s.bits == 32 else torch.uint8
        N._check_buffer("state.exp_avg", s.exp_avg, (end,), (kind,), self.device, False)
        N._check_buffer("state.exp_avg_sq", s.exp_avg_sq, (end,), (kind,), self.device, False)
        if s.bits == 8:
            for name in ("exp_avg_scale", "exp_avg_sq_scale"):
                N._check_buffer("state." + name, getattr(s, name), (end // BLOCK,),
                                (torch.float32,), self.device, False)
        if s.master is not None:
            N._check_buffer("state.master", s.master, (end,), (torch.float32,), self.device, False)

    def _layout(self, kinds, handle=0):
        """The table of tensors for gradients of these types, on the host and the device; made
        again (on the stream of `handle`) when a parameter's storage or decay, the state or a
        gradient's type has changed."""
        import torch
        s = self.state
        each, params, table = torch.Tensor, self.params, self._table
        used = [*params, s.exp_avg, s.exp_avg_sq]
        if s.bits == 8:
            used += (s.exp_avg_scale, s.exp_avg_sq_scale)
        if s.master is not None:
            used.append(s.master)
        pins = list(map(each.data_ptr, used))
        decay = self._weight_decay
        # (a parameter may also have been given another view of the same storage)
        if (table is not None and table[0] == pins and table[1] == kinds and table[2] == decay and
                all(map(each.is_contiguous, params))):
            return table
        decay = list(decay)
        self._check_params()
        self._check_state()
        count, at = len(params), offsets(params)[0]
        rows = (N.AdamWTensor * count)()
        width = 4 if s.bits == 32 else 1
        for i, (p, a) in enumerate(zip(params, at)):
            r = rows[i]
            r.param, r.n = ptr(p), p.numel()
            bf16 = p.dtype == torch.bfloat16
            r.master = s.master.data_ptr() + 4 * a if s.master is not None and bf16 else None
            r.exp_avg = s.exp_avg.data_ptr() + width * a
            r.exp_avg_sq = s.exp_avg_sq.data_ptr() + width * a
            if s.bits == 8:
                r.exp_avg_scale = s.exp_avg_scale.data_ptr() + 4 * (a // BLOCK)
                r.exp_avg_sq_scale = s.exp_avg_sq_scale.data_ptr() + 4 * (a // BLOCK)
            r.weight_decay = decay[i]
            r.param_dtype = dtype_code("params[%d]" % i, p)
            r.grad_dtype = 0 if kinds[i] == torch.bfloat16 else 1
        need = N.nvfp4_adamw_table_bytes(count)
        host = torch.empty(need, dtype=torch.uint8)
        check(N.nvfp4_adamw_table(rows, count, s.bits, host.data_ptr(), need), "nvfp4_adamw_table")
        device = host.to(self.device)
        self._table = (pins, kinds, decay, host, device, host.data_ptr(), device.data_ptr(), handle)
        return self._table

    def _check_grads(self, grads):
        """(pointers, types) of one gradient (or None) per parameter: contiguous, of its shape,
        on its device."""
        import torch
        dev, kinds, each = self.device, (torch.bfloat16, torch.float32), torch.Tensor
        # all at once where all are there and right; otherwise one by one, to say which is not
        try:
            types = [g.dtype for g in grads]
            if (all(map(each.is_contiguous, grads)) and
                    (self._table is not None and types == self._table[1] or set(types).issubset(kinds)) and
                    list(map(each.size, grads)) == self._shapes and
                    list(map(each.get_device, grads)) == [dev.index] * len(types)):
                return self._pack(*map(each.data_ptr, grads)), types
        except (AttributeError, TypeError):
            pass
        for i, (g, shape) in enumerate(zip(grads, self._shapes)):
            if g is None:
                continue
            if g.shape != shape or not g.is_contiguous():
                raise ValueError("grads[%d] must be a contiguous tensor of shape %s" %
                                 (i, tuple(shape)))
            if g.dtype not in kinds:
                raise ValueError("grads[%d] has dtype %s, expected torch.bfloat16 or "
                                 "torch.float32" % (i, g.dtype))
            if g.device != dev:
                raise ValueError("grads[%d] is on %s, expected %s" % (i, g.device, dev))
        # (a missing gradient has the type it had before: the table need not be made again)
        before = self._table[1] if self._table is not None else [p.dtype for p in self.params]
        return (self._pack(*[0 if g is None else g.data_ptr() for g in grads]),
                [t if g is None else g.dtype for g, t in zip(grads, before)])

    def step(self, grads=None, lr=None, grad_scale=None, stream=None):
        """One update.  grads: a list like params (default: each parameter's .grad), contiguous,
        bf16 or float32; None leaves a parameter as it is.  grad_scale: a float32 tensor of one
        element on the GPU that multiplies every gradient (clipping, loss scaling).  lr: this
        step's (and from then on the optimizer's) learning rate."""
        import torch
        if grads is None:
            grads = [p.grad for p in self.params]
        if len(grads) != len(self.params):
            raise ValueError("%d gradients for %d parameters" % (len(grads), len(self.params)))
        dev, f32 = self.device, torch.float32
        pointers, kinds = self._check_grads(grads)   # (pointers: an array, as bytes)
        if grad_scale is not None:
            N._check_buffer("grad_scale", grad_scale.reshape(-1), (1,), (f32,), dev, False)
        if lr is not None:
            self.lr = lr
        s = self.state
        used = () if stream is None else (*grads, grad_scale, *self.params, s.exp_avg, s.exp_avg_sq,
                                          s.exp_avg_scale, s.exp_avg_sq_scale, s.master)

        def call(handle):
            _, _, _, _, table, host, device, home = self._layout(kinds, handle)
            prm = N.AdamWParams(self.lr, self.betas[0], self.betas[1], self.eps, s.step + 1,
                                self.seed, 1 if self.stochastic_rounding else 0, 0,
                                ptr(grad_scale))
            check(N.nvfp4_adamw_step(host, device, pointers, prm, handle), "nvfp4_adamw_step")
            if handle != home:   # (the table may be remade before this stream has passed)
                table.record_stream(torch.cuda.current_stream(dev))
        run_on(stream, dev, used, call)
        torch.autograd.graph.increment_version(self.params)
        s.step += 1

    def moments(self, dtype=None, stream=None):
        """(m, v): the moments' values, flat as the state is; 32-bit moments themselves, 8-bit
        ones decoded to `dtype` (float32 by default, or bf16)."""
        import torch
        s = self.state
        if s.bits == 32:
            return s.exp_avg, s.exp_avg_sq
        dtype = dtype or torch.float32
        if dtype not in (torch.float32, torch.bfloat16):
            raise ValueError("dtype %s, expected torch.bfloat16 or torch.float32" % dtype)
        codes = (s.exp_avg, s.exp_avg_scale, s.exp_avg_sq, s.exp_avg_sq_scale)

        def call(handle):
            m = torch.empty(s.exp_avg.shape, dtype=dtype, device=self.device)
            v = torch.empty(s.exp_avg.shape, dtype=dtype, device=self.device)
            check(N.nvfp4_adamw_moments(ptr(codes[0]), ptr(codes[1]), ptr(codes[2]), ptr(codes[3]),
                                        m.numel(), ptr(m), ptr(v),
                                        1 if dtype == torch.float32 else 0, handle),
                  "nvfp4_adamw_moments")
            return m, v
        return run_on(stream, self.device, codes, call)
