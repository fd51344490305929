"""GPU gated linear recurrence (forward and backward) against binary64, and its hard inputs.

Tolerances, from the operations: with u = 2^-24, sigmoid(g) and 1 - a carry a relative error of
at most d = (16 + 2 |g|) u each (an exponential of |g| log2(e) and a quotient); a step adds
that of its two terms, so the error of h obeys E_t = a_t E_{t-1} + 2 d (a_t |h|_{t-1} +
(1 - a_t) |u_t|) with |h| the recurrence of magnitudes.  However the time axis is split, each
step enters the products once, so the same bound holds.  A bf16 result adds 2^-8 of its
value.  The gradients obey the same recurrence from the end.
"""
import pytest

torch = pytest.importorskip("torch")

from block_scaled_fp4_06_amd import nvfp4 as N  # noqa: E402
from block_scaled_fp4_06_amd import recurrence as R  # noqa: E402

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
BF16, F32, F64 = torch.bfloat16, torch.float32, torch.float64


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


def case(b, t, c, dtype=F32, floor=True, h0=True, docs=0, seed=0):
    g, u = rnd((b, t, c), dtype, seed, 2.0, 2.0), rnd((b, t, c), dtype, seed + 1)
    fl = (0.9 * torch.rand(c, generator=torch.Generator().manual_seed(seed + 2))).cuda() if floor else None
    s = rnd((b, c), F32, seed + 3) if h0 else None
    reset = None
    if docs:
        reset = (torch.rand(b, t, generator=torch.Generator().manual_seed(seed + 4)) < docs / t).cuda()
    return g, u, fl, s, reset


def parts(g, floor, reset):
    """a, 1 - a, sigmoid(g), sigmoid(-g), 1 - floor and the error factor, in binary64."""
    g = g.to(F64)
    lo = torch.zeros(g.shape[2], dtype=F64, device="cuda") if floor is None else floor.to(F64)
    s, sc = 1.0 / (1.0 + torch.exp(-g)), 1.0 / (1.0 + torch.exp(g))
    a, w = lo + (1.0 - lo) * s, (1.0 - lo) * sc
    cut = torch.zeros(g.shape[:2], dtype=torch.bool, device="cuda") if reset is None else reset.bool()
    a, w = a.masked_fill(cut[:, :, None], 0.0), w.masked_fill(cut[:, :, None], 1.0)
    d = (16.0 + 2.0 * g.abs().clamp_max(100.0)) * U
    return a, w, s, sc, 1.0 - lo, d, cut


def close(got, want, tol, what):
    step = 2.0 ** -8 if got.dtype == BF16 else 2 * U
    g = got.detach().to(F64)
    bad = (g - want).abs() > tol + step * want.abs() + 1e-38
    assert not bool(bad.any()), "%s: %d of %d off, worst %.3g" % (
        what, int(bad.sum()), bad.numel(), float(((g - want).abs() - tol).max()))


def check_forward(g, u, floor, h0, reset, **kw):
    y, last = R.gated_scan_forward(g, u, floor, h0, reset, **kw)
    torch.cuda.synchronize()
    b, t, c = g.shape
    a, w, _, _, _, d, _ = parts(g, floor, reset)
    h = torch.zeros((b, c), dtype=F64, device="cuda") if h0 is None else h0.to(F64)
    m, e = h.abs(), torch.zeros_like(h)
    want, tol = torch.empty_like(a), torch.empty_like(a)
    for i in range(t):
        bu = w[:, i] * u[:, i].to(F64)
        e = a[:, i] * e + 2 * d[:, i] * (a[:, i] * m + bu.abs())
        h, m = a[:, i] * h + bu, a[:, i] * m + bu.abs()
        want[:, i], tol[:, i] = h, e
    close(y, want, tol, "y")
    close(last, h, e, "h_last")
    return y, last


def check_backward(dy, g, u, y, floor, h0, reset, dh, **kw):
    got = R.gated_scan_backward(dy, g, u, y, floor, h0, reset, dh, **kw)
    torch.cuda.synchronize()
    b, t, c = g.shape
    a, w, s, sc, rest, d, cut = parts(g, floor, reset)
    grad, tol, size = torch.empty_like(a), torch.empty_like(a), torch.empty_like(a)
    carry = torch.zeros((b, c), dtype=F64, device="cuda") if dh is None else dh.to(F64)
    m, e = carry.abs(), torch.zeros_like(carry)
    for i in reversed(range(t)):
        carry, m = carry + dy[:, i].to(F64), m + dy[:, i].to(F64).abs()
        grad[:, i], size[:, i] = carry, m
        e = e + 2 * U * m
        tol[:, i] = e
        e = a[:, i] * e + 2 * d[:, i] * a[:, i] * m
        carry, m = carry * a[:, i], m * a[:, i]
    first = torch.zeros((b, 1, c), dtype=F64, device="cuda") if h0 is None else h0.to(F64)[:, None]
    before = torch.cat([first, y[:, :-1].to(F64)], 1)
    diff, span = before - u.to(F64), before.abs() + u.to(F64).abs()
    diff, span = (v.masked_fill(cut[:, :, None], 0.0) for v in (diff, span))
    close(got.du, grad * w, tol * w + 2 * d * size * w, "du")
    k = rest * s * sc
    close(got.dg, grad * diff * k, (tol + 4 * d * size) * span * k, "dg")
    close(got.dh0, carry, e, "dh0")
    if floor is None:
        assert got.dfloor is None
    else:
        n = b * t
        close(got.dfloor, (grad * diff * sc).sum((0, 1)),
              ((tol + (4 * d + n * U) * size) * span * sc).sum((0, 1)), "dfloor")
    return got


SIZES = [(1, 1, 1), (3, 1, 70), (2, 2, 8), (1, 7, 3), (2, 65, 16), (1, 300, 65), (3, 257, 24),
         (1, 1000, 200), (2, 2049, 9), (1, 4500, 64), (5, 33, 1000), (70, 5, 40), (1, 3, 5120),
         (1, 1025, 520)]


@pytest.mark.parametrize("b,t,c", SIZES)
@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "fp32"])
def test_sizes(b, t, c, dtype):
    say("scan %dx%dx%d %s" % (b, t, c, dtype))
    g, u, fl, h0, reset = case(b, t, c, dtype, seed=b + t + c)
    y, _ = check_forward(g, u, fl, h0, reset)
    check_backward(rnd((b, t, c), dtype, 8), g, u, y, fl, h0, reset, rnd((b, c), F32, 9))


@pytest.mark.parametrize("floor,h0,docs,dh", [(False, False, 0, False), (True, False, 3, True),
                                              (False, True, 40, False), (False, False, 1e9, True)])
@pytest.mark.parametrize("t,c", [(1, 33), (130, 64), (1300, 40)])
def test_options(floor, h0, docs, dh, t, c):
    say("scan options floor=%s h0=%s docs=%g dh=%s t=%d c=%d" % (floor, h0, docs, dh, t, c))
    g, u, fl, s, reset = case(2, t, c, BF16, floor, h0, docs, seed=t)
    y, _ = check_forward(g, u, fl, s, reset)
    if docs == 1e9:   # every step begins a document: no state at all
        assert torch.equal(y, u)
    check_backward(rnd((2, t, c), BF16, 8), g, u, y, fl, s, reset,
                   rnd((2, c), F32, 9) if dh else None)


def test_reset_as_bytes_and_at_the_edges():
    say("scan resets at the first and last step, as bool and as bytes")
    g, u, fl, h0, _ = case(2, 600, 24, F32)
    reset = torch.zeros((2, 600), dtype=torch.uint8, device="cuda")
    reset[0, 0] = reset[1, 599] = 255
    reset[0, 255:258] = 1
    y, last = check_forward(g, u, fl, h0, reset)
    yb, lb = R.gated_scan_forward(g, u, fl, h0, reset != 0)
    assert torch.equal(y, yb) and torch.equal(last, lb)
    check_backward(rnd((2, 600, 24), F32, 8), g, u, y, fl, h0, reset, rnd((2, 24), F32, 9))


@pytest.mark.parametrize("t,c", [(40, 12), (1500, 64), (1500, 70)])
def test_nothing_passes_a_reset(t, c):
    say("scan: NaN and inf before a reset, t=%d c=%d" % (t, c))
    g, u, fl, h0, _ = case(1, t, c, F32)
    reset = torch.zeros((1, t), dtype=torch.bool, device="cuda")
    cut = t // 2
    reset[0, cut] = True
    bad = [v.clone() for v in (g, u, h0)]
    bad[0][0, 3], bad[1][0, 5, ::2], bad[1][0, cut - 1], bad[2][0, 1] = (
        float("nan"), float("inf"), float("-inf"), float("nan"))
    y, last = R.gated_scan_forward(bad[0], bad[1], fl, bad[2], reset)
    w, lw = R.gated_scan_forward(g, u, fl, h0, reset)
    assert torch.equal(y[:, cut:], w[:, cut:]) and torch.equal(last, lw)
    assert bool(y[0, 3:cut].isnan().all())
    # backward: what follows a reset does not reach what came before it
    dy, dh = rnd((1, t, c), F32, 8), rnd((1, c), F32, 9)
    want = R.gated_scan_backward(dy, g, u, w, fl, h0, reset, dh)
    dy2 = dy.clone()
    dy2[0, cut + 2] = float("nan")
    got = R.gated_scan_backward(dy2, g, u, w, fl, h0, reset, dh)
    assert torch.equal(got.dg[:, :cut], want.dg[:, :cut])
    assert torch.equal(got.du[:, :cut], want.du[:, :cut]) and torch.equal(got.dh0, want.dh0)
    # nor does a NaN state before the reset reach the reset's own gradients
    got = R.gated_scan_backward(dy, bad[0], bad[1], y, fl, bad[2], reset, dh)
    assert torch.equal(got.dg[:, cut:], want.dg[:, cut:])
    assert torch.equal(got.du[:, cut:], want.du[:, cut:])


def test_saturated_gates():
    say("scan: gates of +-inf and beyond the range of exp")
    g, u, fl, h0, _ = case(2, 700, 16, F32)
    g[:, 100:400] = float("inf")    # left out: the state stays
    g[:, 500] = float("-inf")
    g[0, 600], g[1, 600] = 500.0, -500.0
    y, _ = check_forward(g, u, fl, h0, None)
    # (both are within check_forward's bound of the same value, under 100 u of its size each)
    assert float((y[:, 99] - y[:, 399]).abs().max()) <= 200 * U * float(y[:, 99].abs().max())
    d = check_backward(rnd((2, 700, 16), F32, 8), g, u, y, fl, h0, None, rnd((2, 16), F32, 9))
    assert bool((d.du[:, 100:400] == 0).all()) and bool((d.dg[:, 100:400] == 0).all())


@pytest.mark.parametrize("t", [1, 20, 900])
@pytest.mark.parametrize("shift", [0, 1])
def test_halves_of_one_projection(t, shift):
    say("scan of strided halves, t=%d shift=%d" % (t, shift))
    c, dtype = 48, BF16
    both = rnd((3, t, 2 * c + 16), dtype, 1, 2.0)
    g, u = both[:, :, shift:shift + c], both[:, :, c + 8:2 * c + 8]
    _, _, fl, h0, _ = case(3, 1, c, dtype)
    y, last = check_forward(g, u, fl, h0, None)
    yc, lc = R.gated_scan_forward(g.contiguous(), u.contiguous(), fl, h0, None)
    check_backward(rnd((3, t, c), dtype, 8), g, u, y, fl, h0, None, None)
    assert y.shape == yc.shape


def test_time_and_batch_of_zero():
    say("scan of no steps, rows or channels")
    g, u, fl, h0, _ = case(2, 0, 24, F32)
    y, last = R.gated_scan_forward(g, u, fl, h0)
    assert y.shape == (2, 0, 24) and torch.equal(last, h0)
    assert bool((R.gated_scan_forward(g, u)[1] == 0).all())
    dh = rnd((2, 24), F32, 9)
    d = R.gated_scan_backward(g, g, u, y, fl, h0, None, dh)
    assert torch.equal(d.dh0, dh) and bool((d.dfloor == 0).all())
    for b, t, c in ((0, 5, 8), (2, 5, 0)):
        g, u, fl, h0, _ = case(b, t, c, F32)
        y, last = R.gated_scan_forward(g, u, fl, h0)
        d = R.gated_scan_backward(y, g, u, y, fl, h0)
        torch.cuda.synchronize()
        assert y.shape == d.dg.shape == (b, t, c) and bool((d.dfloor == 0).all())


def test_state_kept_in_place_step_by_step():
    say("scan one step at a time, the state in place, against the whole sequence")
    g, u, fl, h0, _ = case(4, 37, 136, F32)
    y, last = R.gated_scan_forward(g, u, fl, h0)
    state = h0.clone()
    for t in range(37):
        yt, s = R.gated_scan_forward(g[:, t:t + 1], u[:, t:t + 1], fl, state, h_last=state)
        assert s is state and float((yt[:, 0] - y[:, t]).abs().max()) <= 64 * U * 8
    assert float((state - last).abs().max()) <= 64 * U * 8


@pytest.mark.parametrize("b,t,c", [(2, 4500, 64), (64, 130, 200), (3, 100, 77), (5, 9, 13)])
def test_long_sequences_keep_the_state_in_place(b, t, c):
    say("scan %dx%dx%d with h_last in h0's place" % (b, t, c))
    g, u, fl, h0, _ = case(b, t, c, BF16)
    y, last = R.gated_scan_forward(g, u, fl, h0)
    for _ in range(3):
        state = h0.clone()
        yi, s = R.gated_scan_forward(g, u, fl, state, h_last=state)
        torch.cuda.synchronize()
        assert s is state and torch.equal(yi, y) and torch.equal(state, last)


def test_continuing_equals_the_whole():
    say("scan in two calls joined by the state")
    g, u, fl, h0, reset = case(2, 1100, 72, F32, docs=4)
    y, last = R.gated_scan_forward(g, u, fl, h0, reset)
    ya, mid = R.gated_scan_forward(g[:, :613], u[:, :613], fl, h0, reset[:, :613].contiguous())
    yb, end = R.gated_scan_forward(g[:, 613:], u[:, 613:], fl, mid, reset[:, 613:].contiguous())
    whole = torch.cat([ya, yb], 1)
    assert float((whole - y).abs().max()) <= 1e-5 and float((end - last).abs().max()) <= 1e-5


def test_offsets_past_32_bits():
    say("scan: time and batch strides past 2^31 elements")
    big = (1 << 31) + 64
    full = torch.empty(2 * big, dtype=BF16, device="cuda")
    g = full.as_strided((2, 20, 64), (big, 64, 1))
    src, u, fl, h0, _ = case(2, 20, 64, BF16)
    g.copy_(src)
    y, last = R.gated_scan_forward(g, u, fl, h0)
    w, lw = R.gated_scan_forward(src, u, fl, h0)
    assert torch.equal(y, w) and torch.equal(last, lw)
    g = full.as_strided((1, 3, 64), (0, big // 2, 1))
    g.copy_(src[:1, :3])
    d = R.gated_scan_backward(u[:1, :3], g, u[:1, :3], y[:1, :3], fl)
    w = R.gated_scan_backward(u[:1, :3], src[:1, :3], u[:1, :3], y[:1, :3], fl)
    assert torch.equal(d.dg, w.dg) and torch.equal(d.dfloor, w.dfloor)


def test_repeats_are_identical():
    say("scan twice: the same bits")
    g, u, fl, h0, reset = case(2, 3000, 200, BF16, docs=3)
    a = [R.gated_scan_forward(g, u, fl, h0, reset) for _ in range(3)]
    dy = rnd((2, 3000, 200), BF16, 8)
    d = [R.gated_scan_backward(dy, g, u, a[0][0], fl, h0, reset) for _ in range(3)]
    torch.cuda.synchronize()
    for k in (1, 2):
        assert torch.equal(a[0][0], a[k][0]) and torch.equal(a[0][1], a[k][1])
        for name in ("dg", "du", "dh0", "dfloor"):
            assert torch.equal(getattr(d[0], name), getattr(d[k], name)), name


@pytest.mark.parametrize("b,t,c", [(24, 2500, 640), (3, 9000, 72)])
@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "fp32"])
def test_a_row_does_not_depend_on_the_others(b, t, c, dtype):
    """More tiles than run at once, each waiting for the state before it."""
    say("scan rows alone %dx%dx%d %s" % (b, t, c, dtype))
    g, u, fl, h0, reset = case(b, t, c, dtype, seed=c)
    dy, dh = rnd((b, t, c), dtype, 8), rnd((b, c), F32, 9)
    y, last = R.gated_scan_forward(g, u, fl, h0, reset)
    d = R.gated_scan_backward(dy, g, u, y, fl, h0, reset, dh)
    for k in (0, b // 2, b - 1):
        row = slice(k, k + 1)
        r = None if reset is None else reset[row]
        y1, last1 = R.gated_scan_forward(g[row], u[row], fl, h0[row], r)
        d1 = R.gated_scan_backward(dy[row], g[row], u[row], y[row], fl, h0[row], r, dh[row])
        torch.cuda.synchronize()
        assert torch.equal(y[row], y1) and torch.equal(last[row], last1)
        for name in ("dg", "du", "dh0"):
            assert torch.equal(getattr(d, name)[row], getattr(d1, name)), name


def test_two_streams_at_once():
    """Tiles of two calls share the GPU; each waits for its own call's tiles only."""
    say("scan on two streams")
    ins = [case(4, 3000, 640, BF16, docs=3, seed=k) for k in (1, 50)]
    want = [R.gated_scan_forward(*i) for i in ins]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in ins]
    got = [[R.gated_scan_forward(*i, stream=s) for i, s in zip(ins, streams)] for _ in range(4)]
    torch.cuda.synchronize()
    for turn in got:
        for (y, last), (y0, last0) in zip(turn, want):
            assert torch.equal(y, y0) and torch.equal(last, last0)


def test_other_stream_and_graph():
    say("scan on another stream and in a HIP graph")
    g, u, fl, h0, reset = case(2, 1500, 128, BF16, docs=3)
    dy = rnd((2, 1500, 128), BF16, 8)
    y, last = R.gated_scan_forward(g, u, fl, h0, reset)
    d = R.gated_scan_backward(dy, g, u, y, fl, h0, reset)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    y2, last2 = R.gated_scan_forward(g, u, fl, h0, reset, stream=s)
    d2 = R.gated_scan_backward(dy, g, u, y2, fl, h0, reset, stream=s)
    s.synchronize()
    assert torch.equal(y, y2) and torch.equal(last, last2) and torch.equal(d.dg, d2.dg)
    assert torch.equal(d.dfloor, d2.dfloor)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y3, last3 = R.gated_scan_forward(g, u, fl, h0, reset)
        d3 = R.gated_scan_backward(dy, g, u, y3, fl, h0, reset)
    for k in range(3):
        u.copy_(rnd(tuple(u.shape), BF16, 40 + k))
        graph.replay()
        torch.cuda.synchronize()
        y, last = R.gated_scan_forward(g, u, fl, h0, reset)
        d = R.gated_scan_backward(dy, g, u, y, fl, h0, reset)
        torch.cuda.synchronize()
        assert torch.equal(y, y3) and torch.equal(last, last3) and torch.equal(d.dg, d3.dg)
        assert torch.equal(d.du, d3.du) and torch.equal(d.dfloor, d3.dfloor)


def test_gradient_against_differences():
    say("scan gradients against differences of the forward pass")
    # the slope of L = sum(y * p) + sum(h_last * q) along a random direction at +-e: truncation
    # O(e^2), rounding about 1e-7 / e of L's terms; at e = 2^-7 both below 5e-3 of the slope
    g, u, fl, h0, reset = case(2, 40, 24, F32, docs=2)
    fl = fl * 0.8 + 0.05
    p, q = rnd((2, 40, 24), F32, 11), rnd((2, 24), F32, 12)
    y, _ = R.gated_scan_forward(g, u, fl, h0, reset)
    d = R.gated_scan_backward(p, g, u, y, fl, h0, reset, q)
    args = [g, u, fl, h0]
    for k, grad in enumerate((d.dg, d.du, d.dfloor, d.dh0)):
        way = rnd(tuple(args[k].shape), F32, 30 + k)
        val = []
        for e in (2.0 ** -7, -2.0 ** -7):
            moved = list(args)
            moved[k] = args[k] + e * way
            yy, ll = R.gated_scan_forward(*moved, reset)
            val.append(float((yy.to(F64) * p.to(F64)).sum() + (ll.to(F64) * q.to(F64)).sum()))
        slope = (val[0] - val[1]) * 64.0
        want = float((grad.to(F64) * way.to(F64)).sum())
        size = float((grad.to(F64) * way.to(F64)).square().sum().sqrt())
        assert abs(slope - want) <= 5e-3 * max(size, abs(want)), (k, slope, want)


def test_autograd():
    say("scan autograd function")
    g, u, fl, h0, reset = case(2, 50, 40, BF16, docs=2)
    leaves = [t.clone().requires_grad_(True) for t in (g, u, fl, h0)]
    y, last = R.autograd_gated_scan().apply(*leaves, reset)
    (y.float().sum() + 3 * last.sum()).backward()
    d = R.gated_scan_backward(torch.ones_like(g), g, u, y.detach(), fl, h0, reset,
                              torch.full((2, 40), 3.0, device="cuda"))
    for t, w in zip(leaves, (d.dg, d.du, d.dfloor, d.dh0)):
        assert torch.equal(t.grad, w)
