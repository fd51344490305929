"""The recurrent block (NVFP4 linears, gated recurrence, norms) and its training example: the
block is the public calls in sequence, its gradients those of a binary32 block up to the
FP4 products' error, a short training run learns, and decoding goes step by step."""
import importlib.util
import os

import pytest

torch = pytest.importorskip("torch")

from block_scaled_fp4_06_amd import block  # noqa: E402
from block_scaled_fp4_06_amd import linear as L  # noqa: E402
from block_scaled_fp4_06_amd import norm  # noqa: E402
from block_scaled_fp4_06_amd import nvfp4 as N  # noqa: E402
from block_scaled_fp4_06_amd import recurrence as R  # noqa: E402

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module", autouse=True)
def gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    N.load()
    yield


def rnd(*shape, seed, std=1.0):
    gen = torch.Generator().manual_seed(seed)
    return (torch.randn(*shape, generator=gen) * std).to(torch.bfloat16).cuda()


def test_block_is_the_calls_in_sequence():
    print("[case] block forward and backward against the single calls", flush=True)
    b, t, d = 2, 72, 96
    p = block.new_block(d, "cuda", seed=3)
    x, h = rnd(b * t, d, seed=1), rnd(b * t, d, seed=2)
    reset = torch.zeros(b, t, dtype=torch.bool, device="cuda")
    reset[1, 40] = True
    x_out, h_next, state, ctx = block.block_forward(x, h, p, b, t, reset=reset, sr_seed=5)
    gu, c1 = L.linear_forward(h, p.w_in, sr_seed=5)
    g, u = gu.view(b, t, -1).split(d, 2)
    y, s = R.gated_scan_forward(g, u, p.floor, None, reset)
    z, c2 = L.linear_forward(y.view(-1, d), p.w_out, sr_seed=7)
    want = norm.residual_norm_forward(x, z, p.post_weight, p.next_weight, p.gate)
    assert torch.equal(x_out, want[0]) and torch.equal(h_next, want[1]) and torch.equal(state, s)
    dx, dh = rnd(b * t, d, seed=8, std=1e-3), rnd(b * t, d, seed=9, std=1e-3)
    got = block.block_backward(dx, dh, ctx)
    n = norm.residual_norm_backward(dx, dh, want[2])
    dy, dw_out = L.linear_backward(n.dz, c2, dw_dtype=torch.bfloat16)
    r = R.gated_scan_backward(dy.view(b, t, d), g, u, y, p.floor, None, reset)
    dh_in, dw_in = L.linear_backward(torch.cat([r.dg, r.du], 2).view(b * t, -1), c1,
                                     dw_dtype=torch.bfloat16)
    assert torch.equal(got[0], n.dx) and torch.equal(got[1], dh_in) and torch.equal(got[2], r.dh0)
    for a, w in zip(got[3].tensors(), (dw_in, dw_out, r.dfloor, n.dpost_weight, n.dgate,
                                       n.dnext_weight)):
        assert torch.equal(a, w)


def test_block_approximates_the_unquantized_block():
    print("[case] block against a binary32 block with autograd", flush=True)
    b, t, d = 4, 64, 128
    p = block.new_block(d, "cuda", seed=4)
    x, h = rnd(b * t, d, seed=1), rnd(b * t, d, seed=2)
    x_out, h_next, _, ctx = block.block_forward(x, h, p, b, t)
    dx, dh = rnd(b * t, d, seed=8, std=1e-3), rnd(b * t, d, seed=9, std=1e-3)
    got = block.block_backward(dx, dh, ctx)
    leaves = [v.detach().float().clone().requires_grad_(True) for v in (x, h, *p.tensors())]
    xf, hf, w_in, w_out, floor, post, gate, nxt = leaves
    g, u = (hf @ w_in).view(b, t, -1).split(d, 2)
    a = floor + (1 - floor) * torch.sigmoid(g)
    state, ys = torch.zeros(b, d, device="cuda"), []
    for i in range(t):
        state = a[:, i] * state + (1 - a[:, i]) * u[:, i]
        ys.append(state)
    z = torch.stack(ys, 1).reshape(b * t, d) @ w_out
    unit = z * torch.rsqrt(z.square().mean(1, keepdim=True) + 1e-6)
    xo = xf + gate * (unit * post)
    ho = xo * torch.rsqrt(xo.square().mean(1, keepdim=True) + 1e-6) * nxt
    (xo * dx.float()).sum().add((ho * dh.float()).sum()).backward()

    def off(a, b):
        return float((a.float() - b).norm() / b.norm())
    # one FP4 product is off by about 0.13 (both operands quantized); a result that goes
    # through k of them by about 0.13 sqrt(k), here at most four, and the norms add bf16
    assert off(x_out, xo.detach()) < 0.2 and off(h_next, ho.detach()) < 0.2
    for a, leaf in zip((got[0], got[1], *got[3].tensors()), leaves):
        assert off(a.view(leaf.shape), leaf.grad) < 0.45, (leaf.shape, off(a.view(leaf.shape), leaf.grad))


def test_training_example_learns_and_decodes():
    print("[case] training example: 80 steps, then decoding", flush=True)
    spec = importlib.util.spec_from_file_location("train_recurrent",
                                                  os.path.join(ROOT, "examples", "train_recurrent.py"))
    ex = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(ex)
    losses, params, head = ex.train(dim=128, blocks=2, batch=16, time=128, steps=80)
    first, last = float(losses[:5].mean()), float(losses[-5:].mean())
    print("  loss %.4f -> %.4f" % (first, last))
    assert bool(losses.isfinite().all()) and last < 0.7 * first
    tokens = rnd(16, 4, 128, seed=6)
    out, states = ex.decode(params, head, tokens, 128)
    torch.cuda.synchronize()
    assert out.shape == (16, 4, 128) and bool(out.isfinite().all())
    assert all(s.shape == (16, 128) for s in states)
