"""GPU recurrent block on a stream that is not the current one."""
import pytest

torch = pytest.importorskip("torch")

from block_scaled_fp4_06_amd import block  # noqa: E402
from block_scaled_fp4_06_amd import nvfp4 as N  # noqa: E402
from test_gpu_block import rnd  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    N.load()
    yield


def busy(stream):
    with torch.cuda.stream(stream):
        torch.cuda._sleep(100000000)


def scribble(sizes):
    """New tensors of these sizes on the current stream, written at once."""
    return [torch.full((n,), 255, dtype=torch.uint8, device="cuda") for n in sizes for _ in range(8)]


def test_block_on_another_stream():
    """Nothing that the block's calls hold between them is handed out on the current stream
    while the other one, kept busy, has not come to them."""
    print("[case] block on another stream", flush=True)
    b, t, d = 2, 72, 96
    p = block.new_block(d, "cuda", seed=3)
    x, h = rnd(b * t, d, seed=1), rnd(b * t, d, seed=2)
    dx, dh = rnd(b * t, d, seed=8, std=1e-3), rnd(b * t, d, seed=9, std=1e-3)
    h0 = torch.randn(b, d, generator=torch.Generator().manual_seed(4)).cuda()
    want = block.block_forward(x, h, p, b, t, h0=h0, sr_seed=5)
    back = block.block_backward(dx, dh, want[3])
    torch.cuda.synchronize()
    sizes = sorted({b * t * d * k // 16 for k in (1, 2, 4, 8, 16, 32, 64, 128)} |
                   {d * d * k // 16 for k in (1, 2, 8, 16, 32, 64)})
    other = torch.cuda.Stream()
    for _ in range(2):
        busy(other)
        got = block.block_forward(x, h, p, b, t, h0=h0, sr_seed=5, stream=other)
        keep = scribble(sizes)
        busy(other)
        gback = block.block_backward(dx, dh, got[3], stream=other)
        keep += scribble(sizes)
        torch.cuda.synchronize()
        assert all(torch.equal(a, w) for a, w in zip(got[:3], want[:3]))
        assert all(torch.equal(a, w) for a, w in zip(gback[:3], back[:3]))
        assert all(torch.equal(a, w) for a, w in zip(gback[3].tensors(), back[3].tensors()))
