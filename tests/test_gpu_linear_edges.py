"""GPU linear layer's autograd function: what it does not do."""
import pytest

torch = pytest.importorskip("torch")

from block_scaled_fp4_06_amd import linear as L  # noqa: E402
from block_scaled_fp4_06_amd import nvfp4 as N  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    N.load()
    yield


def test_second_derivatives_are_refused():
    print("[case] linear: a gradient of a gradient raises", flush=True)
    gen = torch.Generator().manual_seed(1)
    x, w = (torch.randn(64, 64, generator=gen).to(torch.bfloat16).cuda() for _ in range(2))
    x.requires_grad_(True)
    y = L.autograd_linear().apply(x, w, 0, 0)
    g, = torch.autograd.grad(y.float().square().sum(), x, create_graph=True)
    with pytest.raises(RuntimeError, match="once_differentiable"):
        (g.float() * g.float()).sum().backward()


def test_linear_on_another_stream():
    """What lies between the calls is not handed out on the current stream meanwhile."""
    print("[case] linear on another stream", flush=True)
    gen = torch.Generator().manual_seed(2)
    x, w, dy = (torch.randn(*s, generator=gen).to(torch.bfloat16).cuda()
                for s in ((160, 96), (96, 192), (160, 192)))
    y, ctx = L.linear_forward(x, w, sr_seed=3)
    dx, dw = L.linear_backward(dy, ctx)
    torch.cuda.synchronize()
    other = torch.cuda.Stream()
    sizes = [m * n * k // 16 for m, n in ((160, 96), (96, 192), (160, 192)) for k in (1, 8, 32, 64)]
    for _ in range(2):
        with torch.cuda.stream(other):
            torch.cuda._sleep(100000000)
        y2, ctx2 = L.linear_forward(x, w, sr_seed=3, stream=other)
        dx2, dw2 = L.linear_backward(dy, ctx2, stream=other)
        keep = [torch.full((n,), 255, dtype=torch.uint8, device="cuda") for n in sizes for _ in range(8)]
        torch.cuda.synchronize()
        assert torch.equal(y, y2) and torch.equal(dx, dx2) and torch.equal(dw, dw2) and keep
