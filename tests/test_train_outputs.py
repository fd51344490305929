"""Outputs that the caller gives to the operators around the linear layers: what may share
memory and what is refused (no GPU needed)."""
import os

import pytest
import torch

from block_scaled_fp4_06_amd import norm
from block_scaled_fp4_06_amd import nvfp4 as N
from block_scaled_fp4_06_amd import recurrence as R
from block_scaled_fp4_06_amd.launch import apart
from test_train_checks import FAKE, SHAPE, UNSUPPORTED, no_library_calls, sargs, sbackward  # noqa: F401


@pytest.fixture(scope="module", autouse=True)
def lib():
    if not os.path.exists(N.LIB_PATH):
        from block_scaled_fp4_06_amd import build
        build.build()
    return N.load()


def elements(t):
    base = t.data_ptr() // t.element_size()
    at = torch.tensor([base])
    for n, s in zip(t.shape, t.stride()):
        at = (at[:, None] + torch.arange(n) * s).reshape(-1)
    return set(at.tolist())


def test_apart_against_all_elements():
    buf = torch.zeros(4000)
    gen = torch.Generator().manual_seed(1)
    seen = {True: 0, False: 0}
    for _ in range(4000):
        b, t, c, wide = (int(torch.randint(1, n, (1,), generator=gen)) for n in (4, 6, 9, 8))
        st = c + wide
        sb = (t - 1) * st + c + int(torch.randint(0, 12, (1,), generator=gen))
        shape, strides = ((b, t, c), (sb, st, 1)) if wide % 2 else ((t, b, c), (st, sb, 1))
        a, d = (buf.as_strided(shape, strides, 1000 + int(torch.randint(0, 60, (1,), generator=gen)))
                for _ in range(2))
        want = not (elements(a) & elements(d))
        assert apart(a, d) == want, (shape, strides, a.storage_offset(), d.storage_offset())
        seen[want] += 1
    assert min(seen.values()) > 400, seen
    x = torch.zeros(3, 4)
    assert not apart(x, x) and not apart(x, x.t()) and not apart(x, x[1:].view(torch.int32))
    assert apart(x, None) and apart(x[:0], x) and apart(x[:1], x[1:]) and apart(x, x.clone())


def test_scan_gradients_given(no_library_calls):  # noqa: F811
    g = torch.zeros(3, 5, 8)
    both = torch.zeros(3, 5, 16)
    one = torch.zeros(1, 5, 8).expand(3, 5, 8)

    def call(dg, du, **kw):
        a = dict(dy=g.clone(), g=g, u=g.clone(), y=g.clone())
        a.update(kw)
        R.gated_scan_backward(**a, out=(dg, du))
    for dg, du, kw, what in ((one, g.clone(), {}, r"out\[0\] must have rows"),
                             (g.clone(), one, {}, r"out\[1\] must have rows"),
                             (both[:, :, :8], both[:, :, 4:12], {}, "share memory"),
                             (both[:, :, :8], both[:, :, :8], {}, "share memory"),
                             (g, g.clone(), {}, "memory with g"),
                             (g.clone(), both[:, :, 2:10], dict(y=both[:, :, 8:]), "memory with y"),
                             (g.clone(), both[:, :, 8:], dict(h0=both.view(-1)[:24].view(3, 8)), "memory with h0"),
                             (both[:, :, :8], both[:, :, 8:], {}, "GPU"),
                             (both[:, :, 8:], both[:, :, :8], {}, "GPU"),
                             (torch.zeros(5, 3, 8).transpose(0, 1), g.clone(), {}, "GPU"),
                             (g.clone(), g.clone(), dict(dy=one), "GPU")):
        with pytest.raises(ValueError, match=what):
            call(dg, du, **kw)


def test_scan_status_of_outputs():
    far = dict(dg=2 * FAKE, du=3 * FAKE)
    assert sbackward(sargs(), **dict(far, dg_batch=0)) == SHAPE      # rows that overlap
    assert sbackward(sargs(), **dict(far, du_batch=39)) == SHAPE
    assert sbackward(sargs(), **dict(far, dg_batch=8, dg_time=15)) == SHAPE
    assert N.nvfp4_gated_scan_forward(sargs(y_batch=8), FAKE, 1 << 30, None) == SHAPE
    halves = dict(dg_batch=80, dg_time=16, du_batch=80, du_time=16, dg=2 * FAKE)
    for at in (0, 7, -7, 16 + 9, 80 * 2 - 9, 16 * 4 - 1):            # elements from dg
        assert sbackward(sargs(batch=3), du=2 * FAKE + 2 * at, **halves) == UNSUPPORTED, at
    assert sbackward(sargs(), dg=2 * FAKE, du=2 * FAKE + 16, du_time=16, du_batch=80) == UNSUPPORTED


def test_norm_sum_given(no_library_calls):  # noqa: F811
    buf, w = torch.zeros(7, 32), torch.ones(32)
    x, z = buf[:6], torch.zeros(6, 32)
    wide = torch.zeros(6, 64)
    for kw, what in ((dict(out=z), "memory with z"), (dict(out=buf[1:]), "memory with x"),
                     (dict(z=wide[:, 8:40], out=wide[:, :32]), "memory with z"),
                     (dict(gate=wide[:1, :32], out=wide[:, :32]), "memory with gate"),
                     (dict(post_weight=wide[2, 31:63], out=wide[:, :32]), "memory with post_weight"),
                     (dict(z=wide[:, 32:], out=wide[:, :32]), "GPU"),
                     (dict(x=wide[:, 32:], out=wide[:, :32]), "GPU"),
                     (dict(out=x), "GPU"), (dict(out=buf[:6]), "GPU"), (dict(out=torch.zeros(6, 32)), "GPU")):
        with pytest.raises(ValueError, match=what):
            norm.residual_norm_forward(**dict(dict(x=x, z=z, post_weight=w, next_weight=w), **kw))


def test_scan_state_given(no_library_calls):  # noqa: F811
    g, buf = torch.zeros(2, 5, 8), torch.zeros(5, 8)
    h0 = buf[1:3]
    for last, what in ((buf[2:4], "memory with h0"), (buf[:2], "memory with h0"),
                       (g.view(-1)[:16].view(2, 8), "memory with g"), (buf[1:3], "GPU"), (h0, "GPU"),
                       (buf[3:], "GPU"), (torch.zeros(2, 8), "GPU")):
        with pytest.raises(ValueError, match=what):
            R.gated_scan_forward(g, g.clone(), None, h0, h_last=last)
