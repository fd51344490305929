"""When the optimizer's table of tensors is made again, and what it then holds (no GPU needed:
the table is made on the host)."""
import ctypes
import os

import pytest
import torch

from block_scaled_fp4_06_amd import nvfp4 as N
from block_scaled_fp4_06_amd import optim

BF16, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def lib():
    if not os.path.exists(N.LIB_PATH):
        from block_scaled_fp4_06_amd import build
        build.build()
    return N.load()


class Row(ctypes.Structure):
    _fields_ = [("t", N.AdamWTensor), ("first_chunk", ctypes.c_int64)]


def rows(opt, kinds=None):
    """The table's rows as the optimizer would use them for a step now."""
    table = opt._layout([p.dtype for p in opt.params] if kinds is None else kinds)[0]
    head = N.nvfp4_adamw_table_bytes(0)
    return [r.t for r in (Row * len(opt.params)).from_buffer_copy(table.numpy().tobytes()[head:])]


def test_weight_decay_between_steps():
    p = [torch.zeros(300), torch.zeros(5, 5), torch.zeros(7, dtype=BF16)]
    opt = optim.AdamW(p, weight_decay=0.1)
    assert [r.weight_decay for r in rows(opt)] == [0.1] * 3
    table = opt._layout([F32, F32, BF16])[0]
    assert opt._layout([F32, F32, BF16])[0] is table
    opt.weight_decay[1] = 0.0
    assert [r.weight_decay for r in rows(opt)] == [0.1, 0.0, 0.1]
    opt.weight_decay = [0.3, 0.2, 0.1]
    assert [r.weight_decay for r in rows(opt)] == [0.3, 0.2, 0.1]
    opt.weight_decay = 0.5
    assert [r.weight_decay for r in rows(opt)] == [0.5] * 3 and opt.weight_decay == [0.5] * 3
    with pytest.raises(ValueError, match="weight_decay"):
        opt.weight_decay = [0.1]
    assert opt.weight_decay == [0.5] * 3
