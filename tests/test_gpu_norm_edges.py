"""GPU residual norm where its work division has the least to share out.  Tolerances as in
test_gpu_norm."""
import pytest

torch = pytest.importorskip("torch")

from block_scaled_fp4_06_amd import norm  # noqa: E402
from block_scaled_fp4_06_amd import nvfp4 as N  # noqa: E402
from test_gpu_norm import BF16, F32, case, check_backward, check_forward, rnd, say  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    N.load()
    yield


@pytest.mark.parametrize("cols", [7, 8, 64, 257, 512, 1000, 1025, 2048, 2049])
@pytest.mark.parametrize("types", ["bf16", "mixed", "fp32"])
def test_gate_gradient_of_one_row(cols, types):
    """One row: all but one of a workgroup's slots have no rows."""
    say("norm gate gradient of one row, %d cols %s" % (cols, types))
    xt, zt, wt = {"bf16": (BF16, BF16, BF16), "mixed": (F32, BF16, F32), "fp32": (F32, F32, F32)}[types]
    x, z, post, nxt, gate = case(1, cols, xt, zt, wt, seed=cols)
    ctx = check_forward(x, z, post, nxt, gate, branch=0.5)
    dx, dh = rnd((1, cols), xt, 9), rnd((1, cols), zt, 10)
    first = check_backward(ctx, dx, dh)
    assert bool(first.dgate.ne(0).any())
    for _ in range(4):
        again = norm.residual_norm_backward(dx, dh, ctx)
        torch.cuda.synchronize()
        assert torch.equal(again.dgate, first.dgate) and torch.equal(again.dpost_weight, first.dpost_weight)


def test_second_derivatives_are_refused():
    say("norm: a gradient of a gradient raises")
    x, z, post, nxt, gate = case(4, 64, F32, F32, F32)
    x.requires_grad_(True)
    for y in (norm.autograd_residual_norm().apply(x, z, post, nxt, gate, 1.0, 0.5, 1e-6, 0.0)[1],
              norm.autograd_norm().apply(x, nxt, 1e-6, 0.0)):
        g, = torch.autograd.grad(y.square().sum(), x, create_graph=True)
        with pytest.raises(RuntimeError, match="once_differentiable"):
            (g * g).sum().backward()
