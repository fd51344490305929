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


@pytest.mark.parametrize("cols", [5121, 6000, 8192, 8193, 9001, 10240, 16384, 16385, 20481])
@pytest.mark.parametrize("rows,gates", [(1, 1), (9, 3), (300, 1), (300, 6), (260, 260)])
def test_wide_rows(rows, gates, cols):
    """Widths at both ends of every form of the kernels, and the gate rows between slots."""
    say("norm wide rows %dx%d, %d gate rows" % (rows, cols, gates))
    for xt, zt, wt in ((BF16, BF16, F32), (F32, BF16, BF16), (F32, F32, F32)):
        x, z, post, nxt, gate = case(rows, cols, xt, zt, wt, gates, seed=cols + rows)
        ctx = check_forward(x, z, post, nxt, gate, skip=0.9, branch=0.5)
        dx, dh = rnd((rows, cols), xt, 9), rnd((rows, cols), zt, 10)
        d = check_backward(ctx, dx, dh)
        again = norm.residual_norm_backward(dx, dh, ctx)
        torch.cuda.synchronize()
        for name in ("dx", "dz", "dpost_weight", "dnext_weight", "dgate"):
            assert torch.equal(getattr(d, name), getattr(again, name)), name


@pytest.mark.parametrize("cols", [7, 72, 513, 2048, 5120, 6001, 9001])
def test_backward_in_place(cols):
    """dx in dx_out's place and dz in dh's, as the C entry point allows."""
    say("norm backward in place, %d cols" % cols)
    rows = 37
    x, z, post, nxt, gate = case(rows, cols)
    _, _, ctx = norm.residual_norm_forward(x, z, post, nxt, gate)
    dx, dh = rnd((rows, cols), BF16, 9), rnd((rows, cols), BF16, 10)
    want = norm.residual_norm_backward(dx, dh, ctx)
    prm = N.NormParams(rows, cols, 1, 0, 0, 1, 1 if gate.dtype == F32 else 0, 0.0, 0.0, 1.0, 1.0)
    sums = [torch.empty(cols, device="cuda") for _ in range(2)]
    dgate = torch.empty_like(gate)
    need = N.nvfp4_residual_norm_workspace_bytes(prm)
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    p = [t.data_ptr() for t in (ctx.x_out, z, post, gate, nxt, ctx.rstd, ctx.rstd_post, dx, dh, *sums, dgate)]
    args = N.NormBackwardArgs(p[0], cols, p[1], cols, p[2], p[3], cols, p[4], p[5], p[6], p[7], cols, p[8],
                              cols, p[7], cols, p[8], cols, p[9], p[10], p[11], cols)
    assert N.nvfp4_residual_norm_backward(prm, args, ws.data_ptr(), need,
                                          torch.cuda.current_stream().cuda_stream) == N.NVFP4_OK
    torch.cuda.synchronize()
    for got, w in ((dx, want.dx), (dh, want.dz), (sums[0], want.dpost_weight),
                   (sums[1], want.dnext_weight), (dgate, want.dgate)):
        assert torch.equal(got, w)
