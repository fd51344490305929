"""The training-step operators around the NVFP4 linear layers, as measured cases.

Three operators, each in the directions and types a training or serving program uses:

  norm   the norm after a block, its gate and the scaled residual sum, and the norm before
         the next block, forward and backward
  scan   the gated linear recurrence over time, forward (down to one token) and backward
  adamw  one AdamW step over many tensors, moments in 32 or in 8 bits

`own` selects who computes: elementary torch operations in 32 bits (False) or the
library's kernels (True).  `exact` computes the same outputs from the definitions in
binary64.
"""
import math
import random

import torch

own = False

BF16, F32, F64 = torch.bfloat16, torch.float32, torch.float64
DTYPE = {"bf16": BF16, "fp32": F32}
SIZE = {"bf16": 2, "fp32": 4}
EPS = 1e-6
SKIP, BRANCH = 1.0, 0.70710678
BLOCK = 256                     # elements of one 8-bit state block
BETA1, BETA2, ADAM_EPS, LR, DECAY = 0.9, 0.99, 1e-8, 1e-3, 0.1
SEED = 0x5248


# ------------------------------------------------------------------ the cases
def listed():
    return [
        # serving: one token through a block's end and the next block's beginning
        dict(name="norm_one_token", op="norm", way="fwd", rows=1, cols=5120, x="bf16", z="bf16",
             w="bf16", gates=1),
        # training: the repository's activation size, a learned gate per channel
        dict(name="norm_train_fwd", op="norm", way="fwd", rows=8192, cols=5120, x="bf16", z="bf16",
             w="fp32", gates=1),
        dict(name="norm_train_bwd", op="norm", way="bwd", rows=8192, cols=5120, x="bf16", z="bf16",
             w="fp32", gates=1),
        # an odd width, a binary32 residual stream and one gate row per sample
        dict(name="norm_odd_bwd", op="norm", way="bwd", rows=7 * 293, cols=1001, x="fp32",
             z="bf16", w="bf16", gates=7),
        # serving: one token of 64 requests, each with its state
        dict(name="scan_one_token", op="scan", way="fwd", batch=64, time=1, chan=5120, t="bf16",
             docs=0, floor=True),
        # training: 8192 packed tokens of many documents in one row
        dict(name="scan_packed_fwd", op="scan", way="fwd", batch=1, time=8192, chan=5120, t="bf16",
             docs=12, floor=False),
        # training: the same tokens as a batch, with a learned floor of the decay per channel
        dict(name="scan_train_bwd", op="scan", way="bwd", batch=4, time=2048, chan=5120, t="bf16",
             docs=0, floor=True),
        # ragged sizes in binary32
        dict(name="scan_odd_bwd", op="scan", way="bwd", batch=3, time=1021, chan=777, t="fp32",
             docs=4, floor=True),
        # the small tensors of a model: norms, gates, biases
        dict(name="adamw_small", op="adamw", tensors=30, elements=60001, layout=1, p="fp32",
             bits=32, master=False, sr=False),
        # a layer's weights: bf16 with a binary32 master copy and 32-bit moments
        dict(name="adamw_master", op="adamw", tensors=9, elements=5120 * 20480, layout=2, p="bf16",
             bits=32, master=True, sr=False),
        # the same layer with 8-bit moments and stochastically rounded bf16 weights
        dict(name="adamw_8bit", op="adamw", tensors=9, elements=5120 * 20480, layout=2, p="bf16",
             bits=8, master=False, sr=True),
        # many middle-sized tensors, 8-bit moments, binary32 weights
        dict(name="adamw_8bit_many", op="adamw", tensors=60, elements=9000011, layout=3, p="fp32",
             bits=8, master=False, sr=False),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    op = rng.choice(["norm", "norm", "scan", "scan", "adamw", "adamw"])
    if op == "norm":
        cols = _log(rng, 64, 20480)
        cols = cols - cols % 16 if rng.random() < 0.7 and cols >= 64 else cols
        rows = _log(rng, 1, max(1, min(16384, 8192 * 5120 // cols)))
        kind = rng.random()
        if kind < 0.4:
            gates = 1
        elif kind < 0.8:   # one gate row per sample
            gates = rng.randint(1, min(64, rows))
            rows = max(1, rows // gates) * gates
        else:              # one gate row per token
            gates = rows
        x, z = rng.choice([("bf16", "bf16"), ("fp32", "bf16"), ("fp32", "fp32")])
        rows = rows if x == z == "bf16" else max(gates, rows // 2 // gates * gates)
        return dict(op="norm", way=rng.choice(["fwd", "bwd"]), rows=rows, cols=cols, x=x, z=z,
                    w=rng.choice(["bf16", "fp32"]), gates=gates)
    if op == "scan":
        chan = _log(rng, 64, 10240)
        chan = chan - chan % 16 if rng.random() < 0.7 else chan
        t = rng.choice(["bf16", "bf16", "fp32"])
        time = _log(rng, 1, 16384)
        room = 8192 * 5120 // (1 if t == "bf16" else 2) // (chan * time)
        if room < 1:
            time = max(1, time * room if room else 8192 * 5120 // 2 // chan)
            room = 1
        return dict(op="scan", way=rng.choice(["fwd", "bwd"]), batch=_log(rng, 1, min(64, room)),
                    time=time, chan=chan, t=t, docs=rng.choice([0, 3, 20]) if time > 1 else 0,
                    floor=rng.random() < 0.5)
    elements = _log(rng, 20000, 5120 * 20480 // 2)
    p = rng.choice(["bf16", "fp32"])
    return dict(op="adamw", tensors=rng.randint(1, 100), elements=elements,
                layout=rng.randrange(1 << 20), p=p, bits=rng.choice([32, 8]),
                master=p == "bf16" and rng.random() < 0.5, sr=p == "bf16" and rng.random() < 0.5)


def _sizes(case):
    """Element counts of the tensors: of very different sizes, odd ones among them."""
    rng = random.Random(case["layout"])
    parts = [math.exp(rng.gauss(0.0, 1.5)) for _ in range(case["tensors"])]
    scale = case["elements"] / sum(parts)
    return [max(1, int(f * scale)) for f in parts]


def work(case):
    if case["op"] == "norm":
        n, e, s = case["rows"] * case["cols"], SIZE[case["x"]], SIZE[case["z"]]
        par = (2 + case["gates"]) * case["cols"] * SIZE[case["w"]]
        if case["way"] == "fwd":
            return {"bytes": n * (2 * e + 2 * s) + par + 8 * case["rows"], "flops": 12 * n}
        return {"bytes": n * (3 * e + 3 * s) + 2 * par + 8 * case["rows"], "flops": 30 * n}
    if case["op"] == "scan":
        n, e = case["batch"] * case["time"] * case["chan"], SIZE[case["t"]]
        state = case["batch"] * case["chan"] * 4
        marks = case["batch"] * case["time"] if case["docs"] else 0
        if case["way"] == "fwd":
            return {"bytes": n * 3 * e + 2 * state + marks, "flops": 10 * n}
        return {"bytes": n * 6 * e + 3 * state + marks, "flops": 20 * n}
    n, e = sum(_sizes(case)), SIZE[case["p"]]
    # weights in and out (with a master copy they are only written), gradient in
    per = (2 * e if not case["master"] else e + 8) + e
    if case["bits"] == 32:
        per += 16
    else:   # codes in and out and their scales; then the moments as bf16 from the new codes
        per += 4 + 16 / BLOCK + 2 + 8 / BLOCK + 4
    return {"bytes": per * n, "flops": 20 * n}


# ------------------------------------------------------------------ inputs
def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed & 0x7FFFFFFF)


def _normal(gen, *shape):
    return torch.randn(*shape, generator=gen, device="cuda")


def _uniform(gen, *shape):
    return torch.rand(*shape, generator=gen, device="cuda")


def _rows(gen, rows, cols, dtype, std=1.0):
    """Activations: normal, a few channels far larger than the others."""
    x = _normal(gen, rows, cols).mul_(std)
    loud = torch.randint(0, cols, (max(1, cols // 640),), generator=gen, device="cuda")
    x[:, loud] *= 20.0
    return x.to(dtype)


def prepare(case, seed):
    gen = _gen(seed)
    s = {"case": case}
    if case["op"] == "norm":
        r, c, xt, zt, wt = case["rows"], case["cols"], DTYPE[case["x"]], DTYPE[case["z"]], DTYPE[case["w"]]
        s["z"] = _rows(gen, r, c, zt, 0.5)
        s["post"] = (1.0 + 0.1 * _normal(gen, c)).to(wt)
        s["next"] = (1.0 + 0.1 * _normal(gen, c)).to(wt)
        s["gate"] = (0.5 + 0.3 * _normal(gen, case["gates"], c)).to(wt)
        s["x"] = _rows(gen, r, c, xt)    # backward: the stored sum, the next norm's input
        if case["way"] == "bwd":
            s["dx"] = _normal(gen, r, c).mul_(1e-3).to(xt)
            s["dh"] = _normal(gen, r, c).mul_(1e-3).to(zt)
            s["rstd"] = torch.rsqrt(s["x"].float().square().mean(1) + EPS)
            s["rstd_post"] = torch.rsqrt(s["z"].float().square().mean(1) + EPS)
    elif case["op"] == "scan":
        b, t, c, ty = case["batch"], case["time"], case["chan"], DTYPE[case["t"]]
        # decays from a few to some hundred steps long
        s["g"] = _normal(gen, b, t, c).add_(1.0 + 4.0 * _uniform(gen, c)).to(ty)
        s["u"] = _normal(gen, b, t, c).to(ty)
        s["floor"] = 0.9 * _uniform(gen, c) if case["floor"] else None
        s["h0"] = _normal(gen, b, c)
        s["reset"] = _uniform(gen, b, t) < case["docs"] / t if case["docs"] else None
        if case["way"] == "bwd":
            s["dy"] = _normal(gen, b, t, c).mul_(1e-3).to(ty)
            s["dh"] = _normal(gen, b, c).mul_(1e-3)
            s["y"] = _scan_plain(s["g"], s["u"], s["floor"], s["h0"], s["reset"])[0]
    else:
        _prepare_adamw(s, case, gen)
    return s


def _prepare_adamw(s, case, gen):
    """Weights, gradients and moments in flat buffers, each tensor's share from a multiple
    of 256 elements on (the blocks of the 8-bit moments never span two tensors); what lies
    between two tensors is zero."""
    sizes, pt = _sizes(case), DTYPE[case["p"]]
    starts, end = [], 0
    for n in sizes:
        starts.append(end)
        end += -(-n // BLOCK) * BLOCK
    valid = torch.zeros(end, dtype=torch.bool, device="cuda")
    for at, n in zip(starts, sizes):
        valid[at:at + n] = True
    loud = torch.exp2(4.0 * _normal(gen, end // BLOCK, 1)).expand(-1, BLOCK).reshape(-1)
    g = _normal(gen, end).mul_(1e-4).mul_(loud).mul_(valid)
    s["m_start"] = _normal(gen, end).mul_(2e-5).mul_(loud).mul_(valid)
    s["v_start"] = _uniform(gen, end).add_(0.1).mul_(1e-8).mul_(loud.square_()).mul_(valid)
    p = _normal(gen, end).mul_(0.02).mul_(valid)
    s["p"], s["g"] = p.to(pt), g.to(pt)
    s["master"] = p if case["master"] else None
    s["sizes"], s["starts"], s["step"] = sizes, starts, 100
    # biases and gains, the short ones, are not decayed
    s["decay"] = [DECAY if n >= 20000 else 0.0 for n in sizes]
    if case["bits"] == 8:
        m, v = s.pop("m_start"), s.pop("v_start")
        s["mc"], s["ms"] = _m_encode(m.view(-1, BLOCK))
        s["vc"], s["vs"] = _r_encode(v.view(-1, BLOCK).sqrt(), torch.full((1,), 32768, dtype=torch.int64, device="cuda"))
    else:
        s["m"], s["v"] = s.pop("m_start"), s.pop("v_start")
    blocks = [-(-n // BLOCK) for n in sizes]
    count = torch.tensor(blocks, device="cuda")
    s["block_tensor"] = torch.repeat_interleave(torch.arange(len(sizes), device="cuda"), count)
    first = torch.tensor(starts, device="cuda") // BLOCK
    s["block_index"] = torch.arange(end // BLOCK, device="cuda") - first[s["block_tensor"]]
    s["block_decay"] = torch.tensor(s["decay"], dtype=F64, device="cuda")[s["block_tensor"]]
    if own:   # the optimizer object that a training program keeps from step to step
        from block_scaled_fp4_06_amd import optim
        state = optim.AdamWState(
            bits=case["bits"], step=s["step"], master=s["master"],
            exp_avg=s["mc"] if case["bits"] == 8 else s["m"],
            exp_avg_sq=s["vc"] if case["bits"] == 8 else s["v"],
            exp_avg_scale=s["ms"] if case["bits"] == 8 else None,
            exp_avg_sq_scale=s["vs"] if case["bits"] == 8 else None)
        s["params"] = [s["p"][a:a + n] for a, n in zip(starts, sizes)]
        s["grads"] = [s["g"][a:a + n] for a, n in zip(starts, sizes)]
        s["opt"] = optim.AdamW(s["params"], lr=LR, betas=(BETA1, BETA2), eps=ADAM_EPS,
                               weight_decay=s["decay"], state=state,
                               stochastic_rounding=case["sr"], seed=SEED)


# ------------------------------------------------------------------ one pass
def run(s):
    case = s["case"]
    if case["op"] == "norm":
        return _norm_own(s) if own else _norm_plain(s)
    if case["op"] == "scan":
        if own:
            return _scan_own(s)
        if case["way"] == "fwd":
            return _scan_plain(s["g"], s["u"], s["floor"], s["h0"], s["reset"])
        return _scan_bwd_plain(s)
    return _adamw_own(s) if own else _adamw_plain(s)


def _norm_own(s):
    from block_scaled_fp4_06_amd import norm
    if s["case"]["way"] == "fwd":
        x, h, _ = norm.residual_norm_forward(s["x"], s["z"], s["post"], s["next"], gate=s["gate"],
                                             skip_scale=SKIP, branch_scale=BRANCH, eps=EPS)
        return x, h
    ctx = norm.ResidualNormContext(
        x_out=s["x"], z=s["z"], post_weight=s["post"], next_weight=s["next"], gate=s["gate"],
        rstd=s["rstd"], rstd_post=s["rstd_post"], skip_scale=SKIP, branch_scale=BRANCH,
        weight_offset=0.0)
    d = norm.residual_norm_backward(s["dx"], s["dh"], ctx)
    return d.dx, d.dz, d.dpost_weight, d.dnext_weight, d.dgate


def _scan_own(s):
    from block_scaled_fp4_06_amd import recurrence
    if s["case"]["way"] == "fwd":
        return recurrence.gated_scan_forward(s["g"], s["u"], floor=s["floor"], h0=s["h0"],
                                             reset=s["reset"])
    d = recurrence.gated_scan_backward(s["dy"], s["g"], s["u"], s["y"], floor=s["floor"],
                                       h0=s["h0"], reset=s["reset"], dh_last=s["dh"])
    return d.dg, d.du, d.dh0, d.dfloor


def _adamw_own(s):
    opt = s["opt"]
    opt.step(s["grads"])
    if s["case"]["bits"] == 8:
        m, v = opt.moments(torch.bfloat16)
        return s["p"], s["master"], m, v
    return s["p"], s["master"], s["m"], s["v"]


# ------------------------------------------------------------------ plain forms
def _per_row(gate, rows):
    """(G, cols) gate rows, each shared by rows / G consecutive rows."""
    return gate if gate.shape[0] in (1, rows) else gate.repeat_interleave(rows // gate.shape[0], 0)


def _norm_plain(s):
    z, gate = s["z"].float(), _per_row(s["gate"].float(), s["x"].shape[0])
    post, nxt = s["post"].float(), s["next"].float()
    if s["case"]["way"] == "fwd":
        n2 = z * torch.rsqrt(z.square().mean(1, keepdim=True) + EPS)
        x = (SKIP * s["x"].float() + BRANCH * (gate * (n2 * post))).to(s["x"].dtype)
        xf = x.float()
        h = xf * torch.rsqrt(xf.square().mean(1, keepdim=True) + EPS) * nxt
        return x, h.to(s["z"].dtype)
    wt = s["post"].dtype
    r1, r2, dh = s["rstd"][:, None], s["rstd_post"][:, None], s["dh"].float()
    n1, t1 = s["x"].float() * r1, dh * nxt
    d = s["dx"].float() + r1 * (t1 - n1 * (t1 * n1).mean(1, keepdim=True))
    n2 = z * r2
    dp = BRANCH * gate * d
    t2 = dp * post
    dz = r2 * (t2 - n2 * (t2 * n2).mean(1, keepdim=True))
    dgate = (BRANCH * d * (n2 * post)).view(s["gate"].shape[0], -1, d.shape[1]).sum(1)
    return ((SKIP * d).to(s["x"].dtype), dz.to(s["z"].dtype), (dp * n2).sum(0).to(wt),
            (dh * n1).sum(0).to(wt), dgate.to(s["gate"].dtype))


def _decay(g, floor, reset):
    """a, 1 - a, sigmoid(g) and sigmoid(-g) in 32 bits; a = 0 at a reset."""
    sg, sc = torch.sigmoid(g.float()), torch.sigmoid(-g.float())
    a, w = (sg, sc) if floor is None else (floor + (1.0 - floor) * sg, (1.0 - floor) * sc)
    if reset is not None:
        a = torch.where(reset[:, :, None], 0.0, a)
        w = torch.where(reset[:, :, None], 1.0, w)
    return a, w, sg, sc


def _scan(a, b):
    """h_t = a_t h_{t-1} + b_t over dim 1 from h = 0, by doubling spans."""
    span = 1
    while span < a.shape[1]:
        b = torch.cat([b[:, :span], a[:, span:] * b[:, :-span] + b[:, span:]], 1)
        a = torch.cat([a[:, :span], a[:, span:] * a[:, :-span]], 1)
        span *= 2
    return b


def _scan_plain(g, u, floor, h0, reset):
    a, w, _, _ = _decay(g, floor, reset)
    b = w * u.float()
    b[:, 0] += a[:, 0] * h0
    h = _scan(a, b)
    return h.to(g.dtype), h[:, -1].clone()


def _scan_bwd_plain(s):
    a, w, sg, sc = _decay(s["g"], s["floor"], s["reset"])
    dy = s["dy"].to(F32, copy=True)   # (a binary32 input itself must stay as it is)
    dy[:, -1] += s["dh"]
    after = torch.cat([a[:, 1:], torch.zeros_like(a[:, :1])], 1)
    grad = _scan(after.flip(1), dy.flip(1)).flip(1)
    before = torch.cat([s["h0"][:, None], s["y"][:, :-1].float()], 1)
    da = grad * (before - s["u"].float())
    if s["reset"] is not None:
        da = torch.where(s["reset"][:, :, None], 0.0, da)
    dg = da * sg * sc
    dfloor = None
    if s["floor"] is not None:
        dg = dg * (1.0 - s["floor"])
        dfloor = (da * sc).sum((0, 1))
    ty = s["g"].dtype
    return dg.to(ty), (grad * w).to(ty), a[:, 0] * grad[:, 0], dfloor


# 8-bit moments.  First: E4M3 codes times a scale per block.  Second: its root as an unsigned
# float of 4 exponent and 4 mantissa bits, value(c) = 2 f for e = 0 and (16 + f) 2^e
# otherwise (e = c >> 4, f = c & 15).  The scales are powers of two that bring the block's
# largest magnitude into [2^7, 2^8) and [2^18, 2^19).
TINY = 2.0 ** -100


def _scale(top, exponent):
    """Power of two that divides top into [2^exponent, 2^(exponent + 1)); 0 below TINY."""
    two = ((top.view(torch.int32) & 0x7F800000) - (exponent << 23)).view(F32)
    return torch.where(top >= TINY, two, 0.0)


def _m_encode(m):
    scale = _scale(m.abs().amax(1, keepdim=True), 7)
    t = torch.where(scale > 0.0, m / torch.where(scale > 0.0, scale, 1.0), 0.0)
    return t.to(torch.float8_e4m3fn).view(torch.uint8).view(-1), scale.view(-1)


def _m_decode(codes, scale):
    return codes.view(torch.float8_e4m3fn).view(-1, BLOCK).float() * scale[:, None]


def _r_encode(r, draws):
    """draws: 16-bit numbers; the fraction of a step plus (draw + 1/2) / 2^16 carries."""
    scale = _scale(r.amax(1, keepdim=True), 18)
    t = torch.where(scale > 0.0, r / torch.where(scale > 0.0, scale, 1.0), 0.0)
    low = t < 32.0
    bits = torch.where(low, t + 32.0, t).view(torch.int32).to(torch.int64)
    codes = ((bits - 0x42000000 + 8 * draws + 4) >> 19) + torch.where(low, 0, 16)
    codes = torch.where(t > 0.0, codes.clamp(1, 254), 0)
    return codes.to(torch.uint8).view(-1), scale.view(-1)


def _r_decode(codes, scale):
    c = codes.view(-1, BLOCK).to(torch.int32)
    e, f = c >> 4, c & 15
    value = torch.where(e == 0, 2 * f, (16 + f) << e).float()
    return value * scale[:, None]


def _mulhilo(a, b):
    """High and low 32 bits of a * b for a constant a and int64 tensors b < 2^32."""
    low = (a & 0xFFFF) * b
    high = (a >> 16) * b + (low >> 16)
    return (high >> 16) & 0xFFFFFFFF, ((high & 0xFFFF) << 16) | (low & 0xFFFF)


def _draws(s, stream):
    """16-bit draws of every element: lane i % 8 of Philox4x32-10 with counter
    (i / 8, step, 2 tensor + stream), i the element's index in its tensor."""
    eighth = torch.arange(BLOCK // 8, device="cuda")
    i = s["block_index"][:, None] * (BLOCK // 8) + eighth
    c0, c1 = i & 0xFFFFFFFF, i >> 32
    c2 = torch.full_like(i, s["step"])
    c3 = (2 * s["block_tensor"][:, None] + stream).expand_as(i)
    k0, k1 = SEED & 0xFFFFFFFF, SEED >> 32
    for _ in range(10):
        h0, l0 = _mulhilo(0xD2511F53, c0)
        h1, l1 = _mulhilo(0xCD9E8D57, c2)
        c0, c1, c2, c3 = h1 ^ c1 ^ k0, l1, h0 ^ c3 ^ k1, l0
        k0, k1 = (k0 + 0x9E3779B9) & 0xFFFFFFFF, (k1 + 0xBB67AE85) & 0xFFFFFFFF
    words = torch.stack([c0, c1, c2, c3], 2)
    return torch.stack([words & 0xFFFF, words >> 16], 3).view(-1, BLOCK)


def _adamw_scalars(step):
    return LR / (1.0 - BETA1 ** step), 1.0 / math.sqrt(1.0 - BETA2 ** step)


def _adamw_plain(s):
    case = s["case"]
    s["step"] += 1
    rate, root = _adamw_scalars(s["step"])
    g = s["g"].view(-1, BLOCK).float()
    if case["bits"] == 8:
        m, r = _m_decode(s["mc"], s["ms"]), _r_decode(s["vc"], s["vs"])
        v = r * r
    else:
        m, v = s["m"].view(-1, BLOCK), s["v"].view(-1, BLOCK)
    m = BETA1 * m + (1.0 - BETA1) * g
    v = BETA2 * v + (1.0 - BETA2) * (g * g)
    r = torch.sqrt(v)
    p = (s["master"] if case["master"] else s["p"]).view(-1, BLOCK).float()
    keep = (1.0 - LR * s["block_decay"]).float()[:, None]
    p = p * keep - rate * (m / (r * root + ADAM_EPS))
    if case["master"]:
        s["master"].copy_(p.view(-1))
    if case["sr"]:
        p = ((p.view(torch.int32) + _draws(s, 1).to(torch.int32)) & -65536).view(F32)
    s["p"].copy_(p.view(-1).to(s["p"].dtype))
    if case["bits"] == 32:
        s["m"].copy_(m.view(-1))
        s["v"].copy_(v.view(-1))
        return s["p"], s["master"], s["m"], s["v"]
    mc, ms = _m_encode(m)
    vc, vs = _r_encode(r, _draws(s, 0))
    for name, new in (("mc", mc), ("ms", ms), ("vc", vc), ("vs", vs)):
        s[name].copy_(new)
    r = _r_decode(vc, vs)
    return (s["p"], s["master"], _m_decode(mc, ms).view(-1).to(BF16), (r * r).view(-1).to(BF16))


# ------------------------------------------------------------------ binary64
def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "norm":
        return _norm_exact(s)
    if case["op"] == "scan":
        return _scan_exact(s)
    return _adamw_exact(s)


def _norm_exact(s):
    rows, cols = s["x"].shape
    groups = s["gate"].shape[0]
    z, x = s["z"].to(F64), s["x"].to(F64)
    post, nxt, gate = s["post"].to(F64), s["next"].to(F64), s["gate"].to(F64)
    unit = z / torch.sqrt(torch.sum(z * z, 1) / cols + EPS)[:, None]
    if s["case"]["way"] == "fwd":
        gated = (unit * post).view(groups, -1, cols) * gate[:, None]
        total = SKIP * x + BRANCH * gated.view(rows, cols)
        held = total.to(s["x"].dtype).to(F64)   # the next norm reads the stored sum
        return total, held / torch.sqrt(torch.sum(held * held, 1) / cols + EPS)[:, None] * nxt
    dh, dx = s["dh"].to(F64), s["dx"].to(F64)
    norm = torch.sqrt(torch.sum(x * x, 1) / cols + EPS)[:, None]
    into = dh * nxt
    total = dx + into / norm - x * torch.sum(into * x, 1, keepdim=True) / (cols * norm ** 3)
    branch = (BRANCH * total).view(groups, -1, cols)
    dgate = torch.sum(branch * (unit * post).view(groups, -1, cols), 1)
    back = (branch * gate[:, None]).reshape(rows, cols)
    norm2 = torch.sqrt(torch.sum(z * z, 1) / cols + EPS)[:, None]
    through = back * post
    dz = through / norm2 - z * torch.sum(through * z, 1, keepdim=True) / (cols * norm2 ** 3)
    return (SKIP * total, dz, torch.sum(back * unit, 0), torch.sum(dh * x / norm, 0), dgate)


def _scan_exact(s):
    g, u = s["g"].to(F64), s["u"].to(F64)
    low = 0.0 if s["floor"] is None else s["floor"].to(F64)
    gate = 1.0 / (1.0 + torch.exp(-g))
    rest = 1.0 / (1.0 + torch.exp(g))
    a, w = low + (1.0 - low) * gate, (1.0 - low) * rest
    cut = torch.zeros_like(g[:, :, :1]) if s["reset"] is None else s["reset"].to(F64)[:, :, None]
    a, w = a * (1.0 - cut), w * (1.0 - cut) + cut
    times = range(g.shape[1])
    if s["case"]["way"] == "fwd":
        h, b, out = s["h0"].to(F64), w * u, torch.empty_like(g)
        for t in times:
            h = torch.addcmul(b[:, t], a[:, t], h)
            out[:, t] = h
        return out, h
    dy, grad = s["dy"].to(F64), torch.empty_like(g)
    carry = s["dh"].to(F64)
    for t in reversed(times):
        carry = dy[:, t] + carry
        grad[:, t] = carry
        carry = carry * a[:, t]
    before = torch.cat([s["h0"].to(F64)[:, None], s["y"].to(F64)[:, :-1]], 1)
    da = grad * (before - u) * (1.0 - cut)
    dfloor = None if s["floor"] is None else torch.sum(torch.sum(da * rest, 1), 0)
    return da * (1.0 - low) * gate * rest, grad * w, carry, dfloor


def _adamw_exact(s):
    case, step = s["case"], s["step"] + 1
    s["step"] = step
    draws = _draws(s, 1).view(-1) if case["sr"] else None
    draws_v = _draws(s, 0).view(-1) if case["bits"] == 8 else None
    out = [torch.zeros(s["p"].numel(), dtype=F64, device="cuda") for _ in range(4)]
    for start, n, decay in zip(s["starts"], s["sizes"], s["decay"]):
        at = slice(start, start + n)
        g = s["g"][at].to(F64)
        p = (s["p"] if s["master"] is None else s["master"])[at].to(F64)
        if case["bits"] == 8:
            span = slice(start, start + -(-n // BLOCK) * BLOCK)
            blocks = slice(span.start // BLOCK, span.stop // BLOCK)
            m = s["mc"][span].view(torch.float8_e4m3fn).to(F32).to(F64).view(-1, BLOCK)
            m = (m * s["ms"][blocks, None]).view(-1)[:n]
            code = s["vc"][span].to(F64)
            e, f = torch.div(code, 16, rounding_mode="floor"), code % 16
            r = torch.where(e == 0, 2 * f, (16 + f) * torch.pow(2.0, e)).view(-1, BLOCK)
            v = ((r * s["vs"][blocks, None]) ** 2).view(-1)[:n]
        else:
            m, v = s["m"][at].to(F64), s["v"][at].to(F64)
        m = BETA1 * m + (1.0 - BETA1) * g
        v = BETA2 * v + (1.0 - BETA2) * g ** 2
        full = m / (1.0 - BETA1 ** step)
        p = p - LR * decay * p - LR * full / (torch.sqrt(v / (1.0 - BETA2 ** step)) + ADAM_EPS)
        out[1][at] = p
        if case["sr"]:   # 16 dropped bits of the binary32 value against a 16-bit draw
            ulp = torch.exp2(torch.floor(torch.log2(p.abs().clamp_min(1e-38))) - 7)
            p = torch.sign(p) * torch.floor(p.abs() / ulp + draws[at] / 65536.0) * ulp
        out[0][at] = p
        if case["bits"] == 8:
            m, v = _m_round(m), _v_round(v, draws_v[at])
        out[2][at], out[3][at] = m, v
    if s["master"] is None:
        out[1] = None
    return tuple(out)


def _in_blocks(x):
    wide = torch.zeros(-(-x.numel() // BLOCK) * BLOCK, dtype=F64, device="cuda")
    wide[:x.numel()] = x
    return wide.view(-1, BLOCK)


def _unit(b, exponent):
    top = b.abs().amax(1, keepdim=True).clamp_min(1e-300)
    return torch.exp2(torch.floor(torch.log2(top)) - exponent)


def _m_round(m):
    b = _in_blocks(m)
    t = b / _unit(b, 7)
    step = torch.exp2(torch.floor(torch.log2(t.abs().clamp_min(2.0 ** -6))) - 3)
    return (torch.round(t / step) * step * _unit(b, 7)).view(-1)[:m.numel()]


def _v_round(v, draws):
    b = torch.sqrt(_in_blocks(v))
    t = b / _unit(b, 18)
    step = torch.exp2(torch.floor(torch.log2(t.clamp_min(32.0))) - 4)
    up = torch.floor(t / step + (_in_blocks(draws.to(F64)) + 0.5) / 65536.0)
    r = torch.where(t > 0, (up * step).clamp_min(2.0), 0.0) * _unit(b, 18)
    return (r * r).view(-1)[:v.numel()]
