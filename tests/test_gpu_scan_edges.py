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
