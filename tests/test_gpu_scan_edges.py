"""GPU gated recurrence: states kept in place behind resets, saturated gates, the ends of the
work division.  Tolerances as in test_gpu_scan."""
import pytest

torch = pytest.importorskip("torch")

from block_scaled_fp4_06_amd import nvfp4 as N  # noqa: E402
from block_scaled_fp4_06_amd import recurrence as R  # noqa: E402
from test_gpu_scan import BF16, F32, case, say  # noqa: E402

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
