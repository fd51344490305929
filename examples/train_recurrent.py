"""Train a small stack of recurrent blocks on NVFP4 linear layers, then decode with it.

    python examples/train_recurrent.py [--dim 256] [--blocks 2] [--batch 16] [--time 256]
                                       [--steps 200] [--bits 8]

The task: packed rows of noisy walks, a new one beginning at every reset; the target at each
step is the running mean of the walk's inputs so far, mixed over channels by a fixed matrix.
Everything between the data and the loss runs in the library's kernels: norms with gate and
residual sum, NVFP4 linears, the gated recurrence, and one AdamW launch over all parameters
with 8-bit moments and stochastically rounded bf16 weights.
"""
from __future__ import annotations

import argparse
import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import torch  # noqa: E402

from block_scaled_fp4_06_amd import block, norm, optim  # noqa: E402


def batch_of(step, batch, time, dim, device):
    """Inputs, resets and targets of one step."""
    gen = torch.Generator(device=device).manual_seed(1000 + step)
    x = torch.randn(batch, time, dim, generator=gen, device=device)
    reset = torch.rand(batch, time, generator=gen, device=device) < 4.0 / time
    reset[:, 0] = True
    first = torch.where(reset, torch.arange(time, device=device), 0).cummax(1).values
    total = torch.cat([torch.zeros_like(x[:, :1]), x.cumsum(1)], 1)
    since = total[:, 1:] - total.gather(1, first[:, :, None].expand(-1, -1, dim))
    count = torch.arange(time, device=device) - first + 1
    mean = since / count.sqrt()[:, :, None]
    mix = torch.randn(dim, dim, generator=torch.Generator(device=device).manual_seed(5),
                      device=device) * dim ** -0.5
    return x.view(-1, dim).to(torch.bfloat16), reset, (mean @ mix).view(-1, dim)


def forward(x, params, head, batch, time, reset, sr_seed):
    """The stack: (prediction, contexts).  head is the first norm's weight."""
    h, ctx0 = norm.norm_forward(x, head)
    contexts = []
    for k, p in enumerate(params):
        x, h, _, ctx = block.block_forward(x, h, p, batch, time, reset=reset,
                                           sr_seed=sr_seed + 8 * k)
        contexts.append(ctx)
    return h, (ctx0, contexts)


def backward(dh, contexts):
    """Gradients of (head, *blocks' parameters)."""
    ctx0, ctxs = contexts
    dx, grads = None, []
    for ctx in reversed(ctxs):
        dx, dh, _, g = block.block_backward(dx, dh, ctx)
        grads = g.tensors() + grads
    _, dhead = norm.norm_backward(dh, ctx0, dresidual=dx)
    return [dhead] + grads


def train(dim=256, blocks=2, batch=16, time=256, steps=200, bits=8, lr=3e-3, report=None):
    """Losses of every step, and the trained (params, head)."""
    dev = torch.device("cuda:0")
    params = [block.new_block(dim, dev, seed=k) for k in range(blocks)]
    head = torch.ones(dim, device=dev)
    tensors = [head] + [t for p in params for t in p.tensors()]
    # matrices decay, vectors (norms, gates, floors) do not
    decay = [0.01 if t.dim() == 2 and t.shape[0] > 1 else 0.0 for t in tensors]
    opt = optim.AdamW(tensors, lr=lr, betas=(0.9, 0.98), weight_decay=decay, bits=bits,
                      stochastic_rounding=True, seed=7)
    losses = []
    for step in range(steps):
        x, reset, target = batch_of(step, batch, time, dim, dev)
        pred, contexts = forward(x, params, head, batch, time, reset, sr_seed=1000 * step)
        diff = pred.float() - target
        losses.append(diff.square().mean())
        dh = (diff * (2.0 / diff.numel())).to(torch.bfloat16)
        opt.step(backward(dh, contexts), lr=lr * min(1.0, (step + 1) / 20))
        for p in params:   # a decay's floor stays below one
            p.floor.clamp_(0.0, 0.99)
        if report and (step + 1) % report == 0:
            print("step %4d  loss %.4f" % (step + 1, float(torch.stack(losses[-report:]).mean())),
                  flush=True)
    return torch.stack(losses), params, head


def decode(params, head, tokens, dim):
    """One token of each request at a time, the recurrences' states kept between them."""
    requests, time, _ = tokens.shape
    states, outs = [None] * len(params), []
    for t in range(time):
        x = tokens[:, t].contiguous()
        h, _ = norm.norm_forward(x, head)
        for k, p in enumerate(params):
            x, h, states[k], _ = block.block_forward(x, h, p, requests, 1, h0=states[k])
        outs.append(h)
    return torch.stack(outs, 1), states


def main():
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    for name, value in (("dim", 256), ("blocks", 2), ("batch", 16), ("time", 256), ("steps", 200),
                        ("bits", 8)):
        ap.add_argument("--" + name, type=int, default=value)
    a = ap.parse_args()
    losses, params, head = train(a.dim, a.blocks, a.batch, a.time, a.steps, a.bits, report=20)
    print("loss: first 10 steps %.4f, last 10 %.4f" % (float(losses[:10].mean()),
                                                     float(losses[-10:].mean())))
    tokens = torch.randn(16, 8, a.dim, device="cuda").to(torch.bfloat16)
    out, _ = decode(params, head, tokens, a.dim)
    print("decoded", tuple(out.shape))


if __name__ == "__main__":
    main()
