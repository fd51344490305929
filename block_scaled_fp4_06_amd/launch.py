"""What the torch-level calls of norm, recurrence and optim share: the stream a call runs on,
the memory it takes there, and the checks of its tensors."""
from __future__ import annotations

import contextlib

from . import nvfp4 as N

DTYPES = {"torch.bfloat16": 0, "torch.float32": 1}   # nvfp4_dtype


def dtype_code(name, t):
    """nvfp4_dtype of a tensor; ValueError unless it is bf16 or float32."""
    code = DTYPES.get(str(t.dtype))
    if code is None:
        raise ValueError("%s has dtype %s, expected torch.bfloat16 or torch.float32" %
                         (name, t.dtype))
    return code


@contextlib.contextmanager
def on_stream(stream, device, inputs):
    """Run a call on `stream` (None: the current stream of `device`) with `device` current.

    Memory that the call allocates inside belongs to that stream, and the inputs are kept
    from reuse until the stream has passed, so a call on a stream other than the one its
    tensors were made on needs no more from the caller than the order of the work itself.
    Yields the raw stream handle."""
    import torch
    N._require_gpu(device)
    if torch.cuda.current_device() != device.index:
        with torch.cuda.device(device), on_stream(stream, device, inputs) as handle:
            yield handle
        return
    current = torch.cuda.current_stream(device)
    if stream is None or stream == current:
        yield current.cuda_stream
        return
    if stream.device != device:
        raise ValueError("the stream is on %s, the tensors on %s" % (stream.device, device))
    with torch.cuda.stream(stream):
        for t in inputs:
            if t is not None:
                t.record_stream(stream)
        yield stream.cuda_stream


def check(rc, name):
    if rc != N.NVFP4_OK:
        raise N.NVFP4Error(rc, name)


def ptr(t):
    return t.data_ptr() if t is not None and t.numel() else None
