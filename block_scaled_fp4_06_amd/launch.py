"""What the torch-level calls of norm, recurrence and optim share: the stream a call runs on,
the memory it takes there, and the checks of its tensors."""
from __future__ import annotations

from dataclasses import fields, is_dataclass

from . import nvfp4 as N

_CODES = {}


def dtype_code(name, t):
    """nvfp4_dtype of a tensor; ValueError unless it is bf16 or float32."""
    if not _CODES:   # (importing the package needs no torch)
        import torch
        _CODES.update({torch.bfloat16: 0, torch.float32: 1})
    code = _CODES.get(t.dtype)
    if code is None:
        raise ValueError("%s has dtype %s, expected torch.bfloat16 or torch.float32" %
                         (name, t.dtype))
    return code


def run_on(stream, device, inputs, call):
    """call(handle) on `stream` (None: the current stream of `device`) with `device` current.

    Memory that the call allocates belongs to that stream, and the inputs are kept from reuse
    until the stream has passed, so a call on a stream other than the one its tensors were
    made on needs no more from the caller than the order of the work itself."""
    import torch
    N._require_gpu(device)
    index = device.index
    if torch._C._cuda_getDevice() != index:
        with torch.cuda.device(device):
            return run_on(stream, device, inputs, call)
    # (the handle alone: a Stream object costs more than a small call's own work)
    current = torch._C._cuda_getCurrentRawStream(index)
    if stream is None or stream.cuda_stream == current and stream.device == device:
        return call(current)
    if stream.device != device:
        raise ValueError("the stream is on %s, the tensors on %s" % (stream.device, device))
    with torch.cuda.stream(stream):
        for t in inputs:
            if t is not None:
                t.record_stream(stream)
        return call(stream.cuda_stream)


def tensors_in(*parts):
    """The tensors among `parts` and in the fields of their dataclasses."""
    import torch
    for p in parts:
        if isinstance(p, torch.Tensor):
            yield p
        elif is_dataclass(p):
            yield from tensors_in(*(getattr(p, f.name) for f in fields(p)))


def check(rc, name):
    if rc != N.NVFP4_OK:
        raise N.NVFP4Error(rc, name)


def ptr(t):
    """Address of a tensor's first element; 0 (a null pointer) for None and for no elements."""
    return 0 if t is None else t.data_ptr()


def apart(a, b):
    """Whether no element of one tensor shares memory with one of the other.  Tensors whose
    ranges of addresses meet count as sharing unless their strides are the same and rows lie
    apart (the halves of one projection, for example), where the answer is exact."""
    if a is None or b is None or not a.numel() or not b.numel():
        return True
    (a0, a1), (b0, b1) = ((t.data_ptr(), t.data_ptr() + t.element_size() * (1 + sum(
        (n - 1) * s for n, s in zip(t.shape, t.stride())))) for t in (a, b))
    if a1 <= b0 or b1 <= a0:
        return True
    dims = sorted((s, n) for n, s in zip(a.shape, a.stride()) if n > 1)
    if (a.dtype is not b.dtype or (b0 - a0) % a.element_size() or
            dims != sorted((s, n) for n, s in zip(b.shape, b.stride()) if n > 1)):
        return False
    width = 1   # of what the smaller strides span, each beyond the one before
    for s, n in dims:
        if s < width:
            return False
        width += (n - 1) * s

    def meets(d, dims):   # some steps bring the distance d to zero
        if not dims:
            return d == 0
        s, n = dims[-1]
        return any(meets(d + i * s, dims[:-1]) for i in range(-d // s - 1, -d // s + 3) if abs(i) < n)
    return not meets((b0 - a0) // a.element_size(), dims)


def new_like(t):
    """A new contiguous tensor of t's shape and type (None for None)."""
    import torch
    if t is None:
        return None
    return torch.empty_like(t) if t.is_contiguous() else (
        torch.empty(t.shape, dtype=t.dtype, device=t.device))
