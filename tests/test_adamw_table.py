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
    table = opt._layout([p.dtype for p in opt.params] if kinds is None else kinds)[3]
    head = N.nvfp4_adamw_table_bytes(0)
    return [r.t for r in (Row * len(opt.params)).from_buffer_copy(table.numpy().tobytes()[head:])]


def test_weight_decay_between_steps():
    p = [torch.zeros(300), torch.zeros(5, 5), torch.zeros(7, dtype=BF16)]
    opt = optim.AdamW(p, weight_decay=0.1)
    assert [r.weight_decay for r in rows(opt)] == [0.1] * 3
    table = opt._layout([F32, F32, BF16])
    assert opt._layout([F32, F32, BF16]) is table
    opt.weight_decay[1] = 0.0
    assert [r.weight_decay for r in rows(opt)] == [0.1, 0.0, 0.1]
    opt.weight_decay = [0.3, 0.2, 0.1]
    assert [r.weight_decay for r in rows(opt)] == [0.3, 0.2, 0.1]
    opt.weight_decay = 0.5
    assert [r.weight_decay for r in rows(opt)] == [0.5] * 3 and opt.weight_decay == [0.5] * 3
    with pytest.raises(ValueError, match="weight_decay"):
        opt.weight_decay = [0.1]
    assert opt.weight_decay == [0.5] * 3


def test_parameters_replaced_between_steps():
    p = [torch.zeros(300), torch.arange(25.0).view(5, 5)]
    opt = optim.AdamW(p)
    old = [r.param for r in rows(opt)]
    p[1].data = torch.ones(5, 5)
    now = rows(opt)
    assert now[0].param == old[0] and now[1].param == p[1].data_ptr() != old[1] and now[1].n == 25
    p[1].data = p[1].data.to(BF16)
    assert rows(opt)[1].param_dtype == 0
    for data, what in ((p[1].data.t(), r"params\[1\] must be contiguous"),
                       (torch.ones(5, 5).t(), r"params\[1\] must be contiguous"),
                       (torch.ones(25), r"params\[1\] has shape"),
                       (torch.ones(6, 5), r"params\[1\] has shape"),
                       (torch.ones(5, 5).half(), r"params\[1\] has dtype")):
        p[1].data = data
        with pytest.raises(ValueError, match=what):
            rows(opt)
    p[1].data = torch.ones(5, 5)
    assert rows(opt)[1].param == p[1].data_ptr()
    opt.device, p[0].data = torch.device("cuda:0"), torch.zeros(300)   # moved away from its optimizer
    with pytest.raises(ValueError, match=r"params\[0\] is on cpu"):
        rows(opt)


def test_missing_gradients_keep_the_table():
    p = [torch.zeros(300, dtype=BF16), torch.zeros(5, 5, dtype=BF16)]
    opt = optim.AdamW(p)
    grads = [torch.zeros(300), torch.zeros(5, 5, dtype=BF16)]
    table = opt._layout(opt._check_grads(grads)[1])
    assert table[1] == [F32, BF16]
    for missing in ((0,), (1,), (0, 1)):
        some = [None if i in missing else g for i, g in enumerate(grads)]
        assert opt._layout(opt._check_grads(some)[1]) is table, missing
    assert opt._layout(opt._check_grads([None, torch.zeros(5, 5)])[1])[1] == [F32, F32]


def test_parameters_that_share_memory():
    flat = torch.zeros(40)
    a, b = flat[:30], flat[30:]
    optim.AdamW([b, a, torch.zeros(0), flat[:0]])
    for params, what in (([a, torch.zeros(3), a], r"params\[0\] and params\[2\]"),
                         ([b, flat[29:31]], r"params\[0\] and params\[1\]"),
                         ([flat[29:31], a.view(5, 6)], r"params\[0\] and params\[1\]")):
        with pytest.raises(ValueError, match=what + " share memory"):
            optim.AdamW(params)
    opt = optim.AdamW([torch.zeros(30), b])
    rows(opt)
    opt.params[0].data = flat[5:35]
    with pytest.raises(ValueError, match="share memory"):
        rows(opt)
