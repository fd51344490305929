"""GPU residual norm (forward and backward) against binary64, and its hard inputs.

Tolerances, from the operations: u = 2^-24 per binary32 operation; a row's sum of squares is
added in at most 48 dependent steps (up to 32 columns of a thread, then a tree), so a statistic
is off by at most 64 u and an element formed from it by 80 u of the magnitudes it is formed
from; a bf16 result adds half a bf16 step, 2^-8 of its value at most.  h is compared with the
norm of the sum as stored.  A sum over R rows is off by at most (R + 80) u of the sum of its
terms' magnitudes.
"""
import pytest

torch = pytest.importorskip("torch")

from block_scaled_fp4_06_amd import norm  # noqa: E402
from block_scaled_fp4_06_amd import nvfp4 as N  # noqa: E402

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
BF16, F32, F64 = torch.bfloat16, torch.float32, torch.float64
EPS = 1e-6


def say(msg):
    print("[case] " + msg, flush=True)


@pytest.fixture(scope="module", autouse=True)
def gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    N.load()
    yield


def rnd(shape, dtype, seed, std=1.0, mean=0.0):
    gen = torch.Generator().manual_seed(seed)
    return (torch.randn(*shape, generator=gen) * std + mean).to(dtype).cuda()


def step(t):
    return 2.0 ** -8 if t.dtype == BF16 else 2 * U


def close(got, want, scale, what, factor=80):
    """|got - want| <= factor u scale + half a step of the type."""
    g, w = got.detach().to(F64), want
    bad = (g - w).abs() > factor * U * scale + step(got) * w.abs() + 1e-38
    assert not bool(bad.any()), "%s: %d of %d off, worst %.3g" % (
        what, int(bad.sum()), bad.numel(), float(((g - w).abs() / (scale + 1e-38)).max()))


def per_row(gate, rows):
    return gate.to(F64).repeat_interleave(rows // gate.shape[0], 0)


def case(rows, cols, xt=BF16, zt=BF16, wt=F32, gates=1, gt=None, seed=0):
    x, z = rnd((rows, cols), xt, seed), rnd((rows, cols), zt, seed + 1, 0.5)
    post, nxt = rnd((cols,), wt, seed + 2, 0.1, 1.0), rnd((cols,), wt, seed + 3, 0.1, 1.0)
    gate = rnd((gates, cols), gt or wt, seed + 4, 0.3, 0.5) if gates else None
    return x, z, post, nxt, gate


def check_forward(x, z, post, nxt, gate, skip=1.0, branch=1.0, offset=0.0, **kw):
    rows, cols = x.shape
    before = x.to(F64)
    x_out, h, ctx = norm.residual_norm_forward(x, z, post, nxt, gate, skip, branch, EPS, offset, **kw)
    torch.cuda.synchronize()
    assert x_out.dtype == x.dtype and x_out.shape == x.shape
    zf = z.to(F64)
    r2 = 1.0 / torch.sqrt(zf.square().mean(1) + EPS)
    part = zf * r2[:, None] * (offset + post.to(F64)) * branch
    if gate is not None:
        part = part * per_row(gate, rows)
    close(ctx.rstd_post, r2, r2, "rstd_post")
    close(x_out, skip * before + part, (skip * before).abs() + part.abs(), "x_out")
    if nxt is None:
        assert h is None and ctx.rstd is None
        return ctx
    assert h.dtype == z.dtype and h.shape == z.shape
    xf = x_out.to(F64)
    r1 = 1.0 / torch.sqrt(xf.square().mean(1) + EPS)
    want = xf * r1[:, None] * (offset + nxt.to(F64))
    close(ctx.rstd, r1, r1, "rstd")
    close(h, want, want.abs(), "h")
    return ctx


def check_backward(ctx, dx_out, dh, stream=None):
    x, z, gate = ctx.x_out, ctx.z, ctx.gate
    rows, cols = x.shape
    d = norm.residual_norm_backward(dx_out, dh, ctx, stream=stream)
    torch.cuda.synchronize()
    c, zero = ctx.weight_offset, torch.zeros((rows, cols), dtype=F64, device="cuda")
    total, size = zero, zero
    if dx_out is not None:
        total, size = dx_out.to(F64), dx_out.to(F64).abs()
    if dh is not None:
        r = ctx.rstd.to(F64)[:, None]
        n, t = x.to(F64) * r, dh.to(F64) * (c + ctx.next_weight.to(F64))
        total = total + r * (t - n * (t * n).mean(1, keepdim=True))
        size = size + r * (t.abs() + n.abs() * (t * n).abs().mean(1, keepdim=True))
        g = dh.to(F64) * n
        close(d.dnext_weight, g.sum(0), g.abs().sum(0), "dnext_weight", rows + 80)
    else:
        assert d.dnext_weight is None
    close(d.dx, ctx.skip_scale * total, abs(ctx.skip_scale) * size, "dx")
    if z is None:
        assert d.dz is None and d.dpost_weight is None and d.dgate is None
        return d
    rp = ctx.rstd_post.to(F64)[:, None]
    n2, w = z.to(F64) * rp, c + ctx.post_weight.to(F64)
    gt = ctx.branch_scale * (1.0 if gate is None else per_row(gate, rows))
    t2, s2 = gt * w * total, (gt * w).abs() * size if gate is not None else (gt * w.abs()) * size
    close(d.dz, rp * (t2 - n2 * (t2 * n2).mean(1, keepdim=True)),
          rp * (s2 + n2.abs() * (s2 * n2.abs()).mean(1, keepdim=True)), "dz", 160)
    close(d.dpost_weight, (gt * total * n2).sum(0), (size * n2.abs() * abs(gt)).sum(0),
          "dpost_weight", rows + 160)
    if gate is None:
        assert d.dgate is None
    else:
        q = rows // gate.shape[0]
        g = (ctx.branch_scale * total * n2 * w).view(-1, q, cols).sum(1)
        s = (abs(ctx.branch_scale) * size * (n2 * w).abs()).view(-1, q, cols).sum(1)
        close(d.dgate, g, s, "dgate", q + 160)
    return d


SHAPES = [(1, 1), (1, 5120), (2, 7), (3, 64), (33, 257), (5, 1000), (64, 1001), (130, 512),
          (4, 4096), (3, 20480), (2, 32768), (2, 32765), (700, 96), (257, 2056), (1030, 8)]


@pytest.mark.parametrize("rows,cols", SHAPES)
@pytest.mark.parametrize("types", ["bf16", "mixed", "fp32"])
def test_shapes_and_types(rows, cols, types):
    say("norm %dx%d %s" % (rows, cols, types))
    xt, zt, wt = {"bf16": (BF16, BF16, BF16), "mixed": (F32, BF16, F32), "fp32": (F32, F32, F32)}[types]
    x, z, post, nxt, gate = case(rows, cols, xt, zt, wt, seed=rows + cols)
    ctx = check_forward(x, z, post, nxt, gate, branch=0.5)
    check_backward(ctx, rnd((rows, cols), xt, 9), rnd((rows, cols), zt, 10))


@pytest.mark.parametrize("rows,gates", [(12, 1), (12, 2), (12, 12), (600, 3), (600, 300),
                                        (2048, 2048), (1500, 4), (4099, 1)])
@pytest.mark.parametrize("cols", [40, 515])
def test_gates(rows, gates, cols):
    say("norm gates %d of %d rows, %d cols" % (gates, rows, cols))
    x, z, post, nxt, gate = case(rows, cols, BF16, BF16, F32, gates, BF16, seed=gates)
    ctx = check_forward(x, z, post, nxt, gate, skip=0.8, branch=-1.5, offset=1.0)
    check_backward(ctx, rnd((rows, cols), BF16, 9), rnd((rows, cols), BF16, 10))


@pytest.mark.parametrize("cols", [72, 513])
def test_parts_left_out(cols):
    say("norm with parts left out, %d cols" % cols)
    rows = 37
    x, z, post, nxt, gate = case(rows, cols)
    dx, dh = rnd((rows, cols), BF16, 9), rnd((rows, cols), BF16, 10)
    check_backward(check_forward(x, z, post, nxt, None), dx, dh)
    check_backward(check_forward(x, z, post, nxt, gate), None, dh)
    check_backward(check_forward(x, z, post, None, gate), dx, None)
    h, ctx = norm.norm_forward(x, nxt, EPS, 1.0)
    xf = x.to(F64)
    want = xf / torch.sqrt(xf.square().mean(1, keepdim=True) + EPS) * (1.0 + nxt.to(F64))
    close(h, want, want.abs(), "h")
    d = check_backward(ctx, dx, dh)
    a, b = norm.norm_backward(dh, ctx, dresidual=dx)
    assert torch.equal(a, d.dx) and torch.equal(b, d.dnext_weight)
    h, ctx = norm.norm_forward(rnd((3, cols), F32, 4), nxt, out_dtype=BF16)
    assert h.dtype == BF16
    check_backward(ctx, None, rnd((3, cols), BF16, 5))


@pytest.mark.parametrize("cols,ld,at", [(64, 72, 0), (64, 67, 0), (64, 72, 3), (515, 520, 1)])
def test_strides_and_alignment(cols, ld, at):
    say("norm strides: cols %d ld %d first column %d" % (cols, ld, at))
    rows = 19

    def wide(t):
        full = torch.full((rows, ld + at), 7.0, dtype=t.dtype, device="cuda")
        full[:, at:at + cols] = t
        return full[:, at:at + cols]
    x, z, post, nxt, gate = case(rows, cols, gates=rows)
    out = wide(torch.zeros_like(x))
    ctx = check_forward(wide(x), wide(z), post, nxt, wide(gate), out=out)
    base = out._base if out._base is not None else out
    keep = torch.ones(base.shape[1], dtype=torch.bool)
    keep[at:at + cols] = False
    assert bool((base[:, keep.cuda()] == 7.0).all()), "wrote between the rows"
    check_backward(ctx, wide(rnd((rows, cols), BF16, 9)), wide(rnd((rows, cols), BF16, 10)))


def test_in_place():
    say("norm in place")
    x, z, post, nxt, gate = case(50, 200)
    a, ha, _ = norm.residual_norm_forward(x, z, post, nxt, gate)
    version = x._version
    b, hb, _ = norm.residual_norm_forward(x, z, post, nxt, gate, out=x)
    torch.cuda.synchronize()
    assert b is x and x._version > version
    assert torch.equal(a, b) and torch.equal(ha, hb)


def test_empty():
    say("norm of no rows")
    x, z, post, nxt, gate = case(0, 64)
    x_out, h, ctx = norm.residual_norm_forward(x, z, post, nxt, gate)
    assert x_out.shape == h.shape == (0, 64)
    d = norm.residual_norm_backward(x, z, ctx)
    torch.cuda.synchronize()
    assert d.dx.shape == (0, 64)
    for t in (d.dpost_weight, d.dnext_weight, d.dgate):
        assert bool((t == 0).all())
    x, z, post, nxt, gate = case(4, 0)
    x_out, h, ctx = norm.residual_norm_forward(x, z, post, nxt, gate)
    norm.residual_norm_backward(x, z, ctx)
    torch.cuda.synchronize()


@pytest.mark.parametrize("cols", [64, 517])
def test_rows_do_not_touch_each_other(cols):
    say("norm: rows of zeros, inf and NaN, %d cols" % cols)
    x, z, post, nxt, gate = case(9, cols)
    x[1], z[1] = 0, 0
    z[3, 5], x[5, 2], z[7, 0] = float("inf"), float("nan"), float("nan")
    x_out, h, ctx = norm.residual_norm_forward(x, z, post, nxt, gate)
    fine = [0, 1, 2, 4, 6, 8]
    clean = check_forward(x[fine].contiguous(), z[fine].contiguous(), post, nxt, gate)
    assert torch.equal(x_out[fine], clean.x_out) and bool((h[1] == 0).all())
    # z / inf: the row's finite elements vanish, the infinite one is inf / inf
    assert bool(x_out[3].isnan()[5]) and bool(h[5].isnan().all()) and bool(x_out[7].isnan().all())
    d = norm.residual_norm_backward(rnd((9, cols), BF16, 9), rnd((9, cols), BF16, 10), ctx)
    assert bool(d.dx[fine].isfinite().all()) and bool(d.dz[fine].isfinite().all())


def test_large_and_small_magnitudes():
    say("norm of magnitudes 1e15 and 1e-15")
    x, z, post, nxt, gate = case(6, 256, F32, F32, F32)
    z[0] *= 1e15
    z[1] *= 1e-15
    x[2] *= 1e15
    check_backward(check_forward(x, z, post, nxt, gate), rnd((6, 256), F32, 9), rnd((6, 256), F32, 10))


def test_offsets_past_32_bits():
    say("norm: row offsets past 2^32 bytes and 2^31 elements")
    cols, ld = 512, (1 << 31) // 3 + 5
    full = torch.empty(3 * ld + cols, dtype=BF16, device="cuda")
    x = full.as_strided((4, cols), (ld, 1))
    src, z, post, nxt, gate = case(4, cols)
    x.copy_(src)
    ctx = check_forward(x, z, post, nxt, gate)
    assert torch.equal(ctx.x_out, norm.residual_norm_forward(src, z, post, nxt, gate)[0])
    ctx.x_out = x.copy_(ctx.x_out)
    check_backward(ctx, rnd((4, cols), BF16, 9), rnd((4, cols), BF16, 10))


def test_repeats_are_identical():
    say("norm backward twice: the same bits")
    x, z, post, nxt, gate = case(3000, 640)
    _, _, ctx = norm.residual_norm_forward(x, z, post, nxt, gate)
    dx, dh = rnd((3000, 640), BF16, 9), rnd((3000, 640), BF16, 10)
    a, b = (norm.residual_norm_backward(dx, dh, ctx) for _ in range(2))
    torch.cuda.synchronize()
    for name in ("dx", "dz", "dpost_weight", "dnext_weight", "dgate"):
        assert torch.equal(getattr(a, name), getattr(b, name)), name


def test_other_stream():
    say("norm on another stream")
    x, z, post, nxt, gate = case(512, 1024)
    dx, dh = rnd((512, 1024), BF16, 9), rnd((512, 1024), BF16, 10)
    want = norm.residual_norm_forward(x, z, post, nxt, gate)
    dw = norm.residual_norm_backward(dx, dh, want[2])
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    got = norm.residual_norm_forward(x, z, post, nxt, gate, stream=s)
    d = norm.residual_norm_backward(dx, dh, got[2], stream=s)
    s.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    assert torch.equal(d.dz, dw.dz) and torch.equal(d.dpost_weight, dw.dpost_weight)


def test_graph_replay():
    say("norm in a HIP graph, replayed on changing inputs")
    x, z, post, nxt, gate = case(256, 512)
    dx, dh = rnd((256, 512), BF16, 9), rnd((256, 512), BF16, 10)
    norm.residual_norm_backward(dx, dh, norm.residual_norm_forward(x, z, post, nxt, gate)[2])
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        x_out, h, ctx = norm.residual_norm_forward(x, z, post, nxt, gate)
        d = norm.residual_norm_backward(dx, dh, ctx)
    for k in range(3):
        x.copy_(rnd((256, 512), BF16, 20 + k))
        g.replay()
        torch.cuda.synchronize()
        w = norm.residual_norm_forward(x, z, post, nxt, gate)
        dw = norm.residual_norm_backward(dx, dh, w[2])
        torch.cuda.synchronize()
        assert torch.equal(x_out, w[0]) and torch.equal(h, w[1]) and torch.equal(d.dz, dw.dz)
        assert torch.equal(d.dgate, dw.dgate)


def test_gradient_against_differences():
    say("norm gradients against differences of the forward pass")
    # binary64 slope of L = sum(x_out * a + h * b) along a random direction, from the forward
    # kernel at +-e: the truncation error is O(e^2), the rounding error about 1e-7 / e of L's
    # terms; with e = 2^-8 and 6 * 96 terms both stay below 2e-3 of the slope's magnitude
    args = list(case(6, 96, F32, F32, F32, 2))
    a, b = rnd((6, 96), F32, 11).to(F64), rnd((6, 96), F32, 12).to(F64)
    x_out, h, ctx = norm.residual_norm_forward(*args, skip_scale=0.9, branch_scale=1.1)
    d = norm.residual_norm_backward(a.float(), b.float(), ctx)
    grads = (d.dx, d.dz, d.dpost_weight, d.dnext_weight, d.dgate)
    for k, grad in enumerate(grads):
        way = rnd(tuple(args[k].shape), F32, 30 + k)
        val = []
        for e in (2.0 ** -8, -2.0 ** -8):
            moved = list(args)
            moved[k] = args[k] + e * way
            y, g, _ = norm.residual_norm_forward(*moved, skip_scale=0.9, branch_scale=1.1)
            val.append(float((y.to(F64) * a + g.to(F64) * b).sum()))
        slope = (val[0] - val[1]) * 128.0
        want = float((grad.to(F64) * way.to(F64)).sum())
        size = float((grad.to(F64) * way.to(F64)).square().sum().sqrt())
        assert abs(slope - want) <= 2e-3 * max(size, abs(want)), (k, slope, want)


def test_autograd():
    say("norm autograd functions")
    x, z, post, nxt, gate = (t.requires_grad_(True) for t in case(24, 160, gates=3))
    y, h = norm.autograd_residual_norm().apply(x, z, post, nxt, gate, 1.0, 0.5, EPS, 0.0)
    (y.float().sum() + (h.float() * 2).sum()).backward()
    one, two = torch.ones_like(y), torch.full_like(h, 2.0)
    c = [t.detach() for t in (x, z, post, nxt, gate)]
    _, _, ctx = norm.residual_norm_forward(*c, 1.0, 0.5, EPS, 0.0)
    d = norm.residual_norm_backward(one, two, ctx)
    for t, g in zip((x, z, post, nxt, gate),
                    (d.dx, d.dz, d.dpost_weight, d.dnext_weight, d.dgate)):
        assert torch.equal(t.grad, g)
    x2, w2 = c[0].clone().requires_grad_(True), c[3].clone().requires_grad_(True)
    norm.autograd_norm().apply(x2, w2, EPS, 0.0).float().sum().backward()
    _, ctx = norm.norm_forward(c[0], c[3], EPS)
    dx, dw = norm.norm_backward(one, ctx)
    assert torch.equal(x2.grad, dx) and torch.equal(w2.grad, dw)
