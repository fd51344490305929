"""GPU gated recurrence: states kept in place behind resets, saturated gates, the ends of the
work division.  Tolerances as in test_gpu_scan."""
import pytest

torch = pytest.importorskip("torch")

from block_scaled_fp4_06_amd import nvfp4 as N  # noqa: E402
from block_scaled_fp4_06_amd import recurrence as R  # noqa: E402
from test_gpu_scan import BF16, F32, case, check_backward, check_forward, rnd, say  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    N.load()
    yield


@pytest.mark.parametrize("b,t,c", [(1, 4500, 64), (2, 700, 200), (3, 385, 3), (40, 1300, 136)])
@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "fp32"])
def test_state_in_place_behind_resets(b, t, c, dtype):
    """A reset lets the last tile finish without the tiles before it; h0, which the first tile
    still has to read, stays until it has."""
    say("scan in place behind resets %dx%dx%d %s" % (b, t, c, dtype))
    g, u, fl, h0, _ = case(b, t, c, dtype, seed=t)
    for steps in ([t - 130], [t - 1], [128, 256, t - 129, t - 128, t - 127], list(range(0, t, 50)), [0]):
        reset = torch.zeros((b, t), dtype=torch.bool, device="cuda")
        reset[:, steps] = True
        y, last = R.gated_scan_forward(g, u, fl, h0, reset)
        for _ in range(3):
            state = h0.clone()
            yi, s = R.gated_scan_forward(g, u, fl, state, reset, h_last=state)
            torch.cuda.synchronize()
            assert s is state and torch.equal(yi, y) and torch.equal(state, last)


@pytest.mark.parametrize("b,t,c", [(1, 1, 8), (3, 40, 24), (2, 300, 70)])
def test_gradients_given(b, t, c):
    """The halves of one projection's gradient, and time-major tensors: written, and marked so."""
    say("scan gradients given %dx%dx%d" % (b, t, c))
    g, u, fl, h0, reset = case(b, t, c, BF16, docs=2)
    y, _ = R.gated_scan_forward(g, u, fl, h0, reset)
    want = R.gated_scan_backward(u, g, u, y, fl, h0, reset)
    both = torch.full((b, t, 2 * c + 1), 7.0, dtype=BF16, device="cuda")
    turned = [torch.empty((t, b, c), dtype=BF16, device="cuda").transpose(0, 1) for _ in range(2)]
    for dg, du in ((both[:, :, :c], both[:, :, c:-1]), (both[:, :, c:-1], both[:, :, :c]), turned):
        versions = dg._version, du._version
        got = R.gated_scan_backward(u, g, u, y, fl, h0, reset, out=(dg, du))
        torch.cuda.synchronize()
        assert got.dg is dg and torch.equal(dg, want.dg) and torch.equal(du, want.du)
        assert dg._version > versions[0] and du._version > versions[1]
    assert bool((both[:, :, -1] == 7.0).all())


def test_second_derivatives_are_refused():
    say("scan: a gradient of a gradient raises")
    g, u, fl, h0, _ = case(2, 20, 24, F32)
    u.requires_grad_(True)
    y, last = R.autograd_gated_scan().apply(g, u, fl, h0, None)
    d, = torch.autograd.grad(y.square().sum() + last.sum(), u, create_graph=True)
    with pytest.raises(RuntimeError, match="once_differentiable"):
        (d * d).sum().backward()


@pytest.mark.parametrize("t", [16, 17, 128, 300])
@pytest.mark.parametrize("floor", [False, True])
@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "fp32"])
def test_closed_gate_behind_large_states(t, floor, dtype):
    """A gate of -inf gives a = floor exactly, whatever the number of steps."""
    say("scan: gate of -inf behind large states, t=%d floor=%s %s" % (t, floor, dtype))
    c = 70
    g = torch.full((1, t, c), float("inf"), dtype=dtype, device="cuda")   # steps left out
    u = torch.zeros((1, t, c), dtype=dtype, device="cuda")
    fl = torch.linspace(0.0, 0.75, c, device="cuda") if floor else None
    h0 = torch.full((1, c), 3e38, device="cuda")
    h0[0, ::3] = -3e38
    g[0, t // 2] = float("-inf")
    y, last = R.gated_scan_forward(g, u, fl, h0)
    torch.cuda.synchronize()
    want = h0 * fl if floor else torch.zeros_like(h0)
    assert torch.equal(last, want) and torch.equal(y[:, -1], want.to(dtype))
    assert torch.equal(y[:, t // 2 - 1], h0.to(dtype))
    h0[:] = float("inf")   # zero times inf, as by the formula
    y, last = R.gated_scan_forward(g, u, fl, h0)
    torch.cuda.synchronize()
    closed = torch.ones(c, dtype=torch.bool, device="cuda") if fl is None else fl == 0
    assert bool(last[0, closed].isnan().all()) and bool((last[0, ~closed] == float("inf")).all())


@pytest.mark.parametrize("t", [1, 16, 200])
def test_float32_gates_of_any_size(t):
    """1 - a of float32 gates to a few roundings, however large they are: y = (1 - a) u from a
    state of zero at every reset-free first step, here one step per sequence or a reset state.

    Bound (u = 2^-24): exponential 2 u (product's tail, function, factor), 1 + e half, quotient
    2 u, product 1 u: 6 u, twice that with the state's own rounding."""
    say("scan: float32 gates of any size, t=%d" % t)
    c = 4096
    g = torch.zeros((1, t, c), device="cuda")
    g[0, t // 2] = torch.linspace(-86.0, 86.0, c)
    u = torch.zeros((1, t, c), device="cuda")
    u[0, t // 2] = 1.0
    y, _ = R.gated_scan_forward(g, u)
    torch.cuda.synchronize()
    want = 1.0 / (1.0 + torch.exp(g[0, t // 2].double()))
    off = ((y[0, t // 2].double() - want) / want).abs()
    assert float(off.max()) <= 12 * 2.0 ** -24, float(off.max())
    # and a itself, behind a state of one
    g[0], u[0] = float("inf"), 0.0
    g[0, t // 2] = torch.linspace(-86.0, 86.0, c)
    y, last = R.gated_scan_forward(g, u, None, torch.ones((1, c), device="cuda"))
    torch.cuda.synchronize()
    want = 1.0 / (1.0 + torch.exp(-g[0, t // 2].double()))
    off = ((last[0].double() - want) / want).abs()
    assert float(off.max()) <= 12 * 2.0 ** -24, float(off.max())
    d = R.gated_scan_backward(torch.ones_like(y), g, u, y, None, torch.ones((1, c), device="cuda"))
    torch.cuda.synchronize()
    # the gate's step: G = steps from it to the end, du = (1 - a) G
    grad = float(t - t // 2)
    want = grad / (1.0 + torch.exp(g[0, t // 2].double()))
    off = ((d.du[0, t // 2].double() - want) / want).abs()
    assert float(off.max()) <= 12 * 2.0 ** -24, float(off.max())


@pytest.mark.parametrize("b,t,c", [(1, 300, 960), (3, 520, 640), (1, 140, 1000), (31, 17, 64)])
@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "fp32"])
def test_strips_shared_unevenly(b, t, c, dtype):
    """Strips a little fewer than a multiple of eight: some dies have one strip less, and their
    workgroups at its place have none."""
    say("scan strips shared unevenly %dx%dx%d %s" % (b, t, c, dtype))
    g, u, fl, h0, reset = case(b, t, c, dtype, docs=2, seed=c)
    y, _ = check_forward(g, u, fl, h0, reset)
    check_backward(rnd((b, t, c), dtype, 8), g, u, y, fl, h0, reset, rnd((b, c), F32, 9))


def test_more_strips_and_tiles_than_one_launch_takes():
    say("scan of more strips and tiles than one launch takes")
    b, t, c = (1 << 20) + 9, 1100, 1   # 9 tiles a strip: launches of 8, twice
    gen = torch.Generator(device="cuda").manual_seed(1)
    g, u = (torch.randn(b, t, c, generator=gen, device="cuda", dtype=BF16) for _ in range(2))
    h0 = torch.randn(b, c, generator=gen, device="cuda")
    y, last = R.gated_scan_forward(g, u, None, h0)
    d = R.gated_scan_backward(u, g, u, y, None, h0, None, h0)
    torch.cuda.synchronize()
    for first, end in ((0, 5), ((1 << 20) - 3, b), (777777, 777790)):
        rows = slice(first, end)
        y1, last1 = R.gated_scan_forward(g[rows], u[rows], None, h0[rows])
        d1 = R.gated_scan_backward(u[rows], g[rows], u[rows], y1, None, h0[rows], None, h0[rows])
        torch.cuda.synchronize()
        assert torch.equal(y[rows], y1) and torch.equal(last[rows], last1)
        for name in ("dg", "du", "dh0"):
            assert torch.equal(getattr(d, name)[rows], getattr(d1, name)), name
