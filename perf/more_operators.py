"""What the feed-forward operators over block-quantized weights are measured on: the gated block
(both projections, the activation and the product), the projection with bias, activation and
residual in its epilogue, and the backward passes of both to their inputs.

Each case is one pass of one operator.  `run` computes it either in its plain form (torch
operations in 32 bits, rounded once at the end) or, where `own` is true, through the package's
public functions.  `exact` computes it in 64 bits from the definition.

    project           z = x W^T + bias,  y = act(z) + residual          (pre: z, where wanted)
    gated             g = x Wg^T + bg,  u = x Wu^T + bu,  h = act(g) u  (gate, up: g and u, where wanted)
    project_backward  dz = dy act'(z),  dx = dz W
    gated_backward    dg = dh u act'(g),  du = dh act(g),  dx = dg Wg + du Wu

The rows enter as they are, in f32, bf16 or f16; the weights are Q8_0, Q4_K, Q5_K or Q6_K blocks,
frozen: what a weight stands for is a product of its code and its block's scales.
"""
import math

import torch

own = False

# bytes of a block and its values
BLOCK = {"q8_0": (34, 32), "q4_k": (144, 256), "q5_k": (176, 256), "q6_k": (210, 256)}
DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


# ---------------------------------------------------------------------------------------- cases
def listed():
    """Widths are those of this repository's 7B GQA layer (3584 wide, 18944 in the feed-forward block,
    512 for the keys) and of its experts (768 x 2048) unless a comment says otherwise."""
    def case(name, op, fmt, dtype, rows, N, K, act, bias=False, residual=False, save=False):
        return dict(name=name, op=op, fmt=fmt, dtype=dtype, rows=rows, N=N, K=K, act=act, bias=bias, residual=residual,
                    save=save)
    return [
        # one user's next token through the first half of the feed-forward block
        case("gated_one", "gated", "q4_k", "bf16", 1, 18944, 3584, "silu"),
        # the next tokens of a serving batch
        case("gated_batch", "gated", "q6_k", "f16", 48, 18944, 3584, "silu"),
        # a prompt of 2048 tokens: the largest
        case("gated_prompt", "gated", "q4_k", "bf16", 2048, 18944, 3584, "silu"),
        # one expert's share of a training batch in f32, with biases, what the backward pass needs kept
        case("gated_f32", "gated", "q8_0", "f32", 777, 768, 2048, "gelu_tanh", bias=True, save=True),
        # the key projection of one token, with its bias: the smallest call, where latency counts
        case("project_one", "project", "q8_0", "f32", 1, 512, 3584, "none", bias=True),
        # the second half of the feed-forward block, into the residual stream, a few users' next tokens
        case("project_batch", "project", "q6_k", "bf16", 9, 3584, 18944, "none", residual=True),
        # the same for a prompt
        case("project_prompt", "project", "q4_k", "f16", 2048, 3584, 18944, "none", residual=True),
        # a plain two-layer block's first half in f32, a prompt of an odd length
        case("project_f32", "project", "q5_k", "f32", 517, 3584, 3584, "gelu", bias=True),
        # adapters trained over the frozen block: a batch of 2048 tokens back through it
        case("gated_backward_batch", "gated_backward", "q4_k", "bf16", 2048, 18944, 3584, "silu", save=True),
        # the expert's share of the batch back, in f32
        case("gated_backward_f32", "gated_backward", "q8_0", "f32", 777, 768, 2048, "gelu_tanh", save=True),
        # a short sequence back through the second half
        case("project_backward_short", "project_backward", "q6_k", "f16", 133, 3584, 18944, "none"),
        # and through a square projection with an activation, its own gradient kept for an adapter
        case("project_backward_act", "project_backward", "q5_k", "bf16", 1030, 3584, 3584, "relu", save=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    """One more case: single tokens, batches and prompts, forward and backward, over the ranges of the
    listed ones."""
    op = rng.choice(["gated", "gated", "project", "project", "gated_backward", "project_backward"])
    fmt = rng.choice(["q8_0", "q4_k", "q5_k", "q6_k"])
    most = 2048 * 18944 * 3584 * (1 if op.startswith("gated") else 2)  # rows * N * K of the largest listed
    unit = 32 if fmt == "q8_0" else 256
    while True:
        rows = rng.choice([1, rng.randint(2, 16), _log(rng, 16, 256), _log(rng, 256, 2048)])
        N = _log(rng, 64, 18944)
        K = unit * max(1, _log(rng, 256, 18944) // unit)
        if rng.random() < 0.5:
            N, K = rng.choice([(18944, 3584), (3584, 18944), (3584, 3584), (512, 3584), (768, 2048)])
        dtype = rng.choice(["f32", "bf16", "f16"])
        if rows * N * K * (3 if dtype == "f32" else 1) <= most and N * K <= 18944 * 3584 and rows * N * K >= 1 << 16:
            break
    backward = op.endswith("backward")
    return dict(op=op, fmt=fmt, dtype=dtype, rows=rows, N=N, K=K,
                act=rng.choice(["none", "silu", "silu", "gelu", "gelu_tanh", "relu"]),
                bias=not backward and rng.random() < 0.4, residual=op == "project" and rng.random() < 0.5,
                save=rng.random() < 0.4)


def _row_bytes(fmt, K):
    nbytes, values = BLOCK[fmt]
    return K // values * nbytes


def work(case):
    """Weights and rows in, outputs out, each once; two operations for each weight and row."""
    M, N, K, op = case["rows"], case["N"], case["K"], case["op"]
    e = 4 if case["dtype"] == "f32" else 2
    mats = 2 if op.startswith("gated") else 1
    nbytes = mats * N * _row_bytes(case["fmt"], K)
    if op.endswith("backward"):
        pre = mats if op == "gated_backward" or case["act"] != "none" else 0
        nbytes += M * K * e + M * N * e * (1 + pre + (mats if case["save"] else 0))
    else:
        nbytes += M * K * e + M * N * e * (1 + case["residual"] + (mats if case["save"] else 0))
        nbytes += mats * N * 4 if case["bias"] else 0
    return {"bytes": nbytes, "flops": 2 * mats * M * N * K}


# ---------------------------------------------------------------------------------------- inputs
def _half_bytes(x):
    return x.to(torch.float16).contiguous().view(torch.uint8).view(*x.shape, 2)


def _weights(fmt, N, K, gen):
    """Blocks as quantized normal weights of deviation 0.02 have them: uint8 [N, row bytes]."""
    dev = gen.device
    nbytes, values = BLOCK[fmt]
    nb = K // values
    out = torch.empty((N, nb, nbytes), dtype=torch.uint8, device=dev)
    step = max(1, (1 << 26) // K)
    for i in range(0, N, step):
        n = min(step, N - i)
        x = torch.randn((n, nb, values), device=dev, generator=gen)
        spread = torch.rand((n, nb, 1), device=dev, generator=gen) * 0.6 + 0.7  # of the block's deviation
        part = out[i:i + n]
        if fmt == "q8_0":
            top = x.abs().amax(-1, keepdim=True)
            part[..., :2] = _half_bytes((top * spread * (0.02 / 127))[..., 0])
            part[..., 2:] = (x * (127 / top)).round().to(torch.int8).view(torch.uint8)
        elif fmt == "q6_k":
            sub = torch.randint(70, 128, (n, nb, 16), device=dev, generator=gen)
            sub = torch.where(torch.rand((n, nb, 16), device=dev, generator=gen) < 0.5, sub, -sub)
            q = (x * 9.5).round().add_(32).clamp_(0, 63).to(torch.uint8).view(n, nb, 2, 4, 32)
            low, high = q & 15, q >> 4
            part[..., :128] = (low[..., 0:2, :] | low[..., 2:4, :] << 4).reshape(n, nb, 128)
            part[..., 128:192] = (high[..., 0, :] | high[..., 1, :] << 2 | high[..., 2, :] << 4 | high[..., 3, :] << 6
                                  ).reshape(n, nb, 64)
            part[..., 192:208] = sub.to(torch.int8).view(torch.uint8)
            part[..., 208:] = _half_bytes((spread * (0.02 / 9.5 / 100))[..., 0])
        else:
            top = 15 if fmt == "q4_k" else 31
            sub = torch.randint(35, 64, (n, nb, 8), device=dev, generator=gen)
            mins = torch.randint(35, 64, (n, nb, 8), device=dev, generator=gen)
            part[..., 0:2] = _half_bytes((spread * (0.02 * 4.6 / top / 50))[..., 0])
            part[..., 2:4] = _half_bytes((spread * (0.02 * 2.3 / 50))[..., 0])
            part[..., 4:8] = (sub[..., :4] | sub[..., 4:] >> 4 << 6).to(torch.uint8)
            part[..., 8:12] = (mins[..., :4] | mins[..., 4:] >> 4 << 6).to(torch.uint8)
            part[..., 12:16] = (sub[..., 4:] & 15 | (mins[..., 4:] & 15) << 4).to(torch.uint8)
            q = (x * (top / 4.6)).add_(top / 2).round_().clamp_(0, top).to(torch.uint8).view(n, nb, 4, 2, 32)
            if fmt == "q5_k":
                bits = q >> 4  # [n, nb, 4, 2, 32]
                shift = torch.arange(8, device=dev, dtype=torch.uint8).view(4, 2, 1)
                part[..., 16:48] = (bits << shift).sum((-3, -2)).to(torch.uint8)
                q = q & 15
            part[..., nbytes - 128:] = (q[..., 0, :] | q[..., 1, :] << 4).reshape(n, nb, 128)
    return out.view(N, nb * nbytes)


def prepare(case, seed):
    """Weights as loaded, the rows as slices of wider buffers where that is how they come."""
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev).manual_seed(int(seed))
    M, N, K, dt, op = case["rows"], case["N"], case["K"], DTYPES[case["dtype"]], case["op"]

    def rand(rows, width, by=1.0):
        return (torch.randn((rows, width), device=dev, generator=gen) * by).to(dt)
    s = dict(case=case, weights=[_weights(case["fmt"], N, K, gen) for _ in range(2 if op.startswith("gated") else 1)],
             pre=[], bias=[None, None], residual=None)
    if op.endswith("backward"):
        # gradients fall off from token to token; pre-activations as the forward pass leaves them
        fall = torch.rand((M, 1), device=dev, generator=gen).mul_(6.0).neg_().exp_() * 1e-3
        s["grad"] = (torch.randn((M, N), device=dev, generator=gen) * fall).to(dt)
        if op == "gated_backward" or case["act"] != "none":
            s["pre"] = [rand(M, N, 1.2) for _ in s["weights"]]
    else:
        s["x"] = rand(M, K)
        if case["bias"]:
            s["bias"] = [torch.randn((N,), device=dev, generator=gen) * 0.1 for _ in s["weights"]]
        if case["residual"]:
            s["residual"] = rand(M, N, 2.0)
    return s


# ----------------------------------------------------------------------------------- plain forms
def _values(fmt, w):
    """f32 values [N, K] of blocks uint8 [N, row bytes]."""
    nbytes, values = BLOCK[fmt]
    N = w.shape[0]
    b = w.view(N, -1, nbytes)

    def half(at):
        return b[..., at:at + 2].contiguous().view(torch.float16).float()
    if fmt == "q8_0":
        return (b[..., 2:].contiguous().view(torch.int8).float() * half(0)).view(N, -1)
    if fmt == "q6_k":
        low, high = b[..., :128].view(N, -1, 2, 2, 32), b[..., 128:192].view(N, -1, 2, 1, 32)
        low = torch.cat((low & 15, low >> 4), -2)  # [N, nb, 2, 4, 32]
        high = torch.cat([(high >> i) & 3 for i in (0, 2, 4, 6)], -2)
        q = (low | high << 4).view(N, -1, 16, 16).float() - 32.0
        scale = b[..., 192:208].contiguous().view(torch.int8).float() * half(208)
        return (q * scale[..., None]).view(N, -1)
    s = b[..., 4:16].to(torch.int32)
    sub = torch.cat((s[..., :4] & 63, s[..., 8:] & 15 | s[..., :4] >> 6 << 4), -1).float()
    mins = torch.cat((s[..., 4:8] & 63, s[..., 8:] >> 4 | s[..., 4:8] >> 6 << 4), -1).float()
    q = b[..., nbytes - 128:].view(N, -1, 4, 1, 32)
    q = torch.cat((q & 15, q >> 4), -2).view(N, -1, 8, 32)
    if fmt == "q5_k":
        bits = b[..., 16:48].view(N, -1, 1, 32)
        q = q | torch.cat([(bits >> i & 1) << 4 for i in range(8)], -2)
    return (q.float() * (sub * half(0))[..., None] - (mins * half(2))[..., None]).view(N, -1)


def _act(name, z):
    """The activation and its derivative."""
    if name == "none":
        return z, torch.ones_like(z)
    if name == "relu":
        return z.clamp(min=0), (z > 0).to(z.dtype)
    if name == "silu":
        p = 1 / (1 + torch.exp(-z))
        return z * p, p * (1 + z * (1 - p))
    if name == "gelu":
        p = 0.5 * (1 + torch.erf(z * math.sqrt(0.5)))
        return z * p, p + z * torch.exp(-0.5 * z * z) / math.sqrt(2 * math.pi)
    c, a = math.sqrt(2 / math.pi), 0.044715
    p = 1 / (1 + torch.exp(-2 * c * (z + a * z * z * z)))  # (1 + tanh) / 2
    return z * p, p + 2 * z * p * (1 - p) * c * (1 + 3 * a * z * z)


def _plain(s):
    c = s["case"]
    op, act = c["op"], c["act"]
    dt = DTYPES[c["dtype"]]
    if op.endswith("backward"):
        dy = s["grad"].float()
        if op == "gated_backward":
            g, u = (p.float() for p in s["pre"])
            a, da = _act(act, g)
            dz = [dy * u * da, dy * a]
        else:
            dz = [dy * _act(act, s["pre"][0].float())[1] if s["pre"] else dy]
        dx = None
        for d, w in zip(dz, s["weights"]):
            p = torch.matmul(d, _values(c["fmt"], w))
            dx = p if dx is None else dx.add_(p)
        return [dx.to(dt)] + [d.to(dt) for d in dz if c["save"]]
    x = s["x"].float()
    z = []
    for w, b in zip(s["weights"], s["bias"]):
        p = torch.matmul(x, _values(c["fmt"], w).T)
        z.append(p if b is None else p.add_(b))
    y = _act(act, z[0])[0]
    if op == "gated":
        y = y * z[1]
    elif s["residual"] is not None:
        y = y + s["residual"].float()
    return [y.to(dt)] + [p.to(dt) for p in z if c["save"]]


def run(state):
    s, c = state, state["case"]
    if not own:
        return _plain(s)
    import block_quantized_int8_mmq_gb300 as mmq
    fmt, act, w = c["fmt"], c["act"], s["weights"]
    if c["op"] == "gated":
        kept = [torch.empty((c["rows"], c["N"]), dtype=s["x"].dtype, device="cuda") for _ in w] if c["save"] else []
        gate, up = kept or (None, None)
        h = mmq.mmq_gated(s["x"], w[0], w[1], fmt, c["N"], act=act, bias_gate=s["bias"][0], bias_up=s["bias"][1],
                          gate=gate, up=up)
        return [h] + kept
    if c["op"] == "project":
        kept = [torch.empty((c["rows"], c["N"]), dtype=s["x"].dtype, device="cuda")] if c["save"] else []
        y = mmq.mmq_project(s["x"], w[0], fmt, c["N"], bias=s["bias"][0], act=act, residual=s["residual"],
                            pre=kept[0] if kept else None)
        return [y] + kept
    kept = [torch.empty_like(s["grad"]) for _ in w] if c["save"] else []
    if c["op"] == "gated_backward":
        dgate, dup = kept or (None, None)
        dx = mmq.mmq_gated_backward(s["grad"], s["pre"][0], s["pre"][1], w[0], w[1], fmt, c["K"], act=act, dgate=dgate,
                                    dup=dup)
    else:
        dx = mmq.mmq_project_backward(s["grad"], w[0], fmt, c["K"], act=act, pre=s["pre"][0] if s["pre"] else None,
                                      dz=kept[0] if kept else None)
    return [dx] + kept


# ------------------------------------------------------------------------------------- 64 bits
def _table(fmt):
    """For each value of a block: the byte of its low bits and their shift, the byte of its high bits
    and their shift, its group of equal scales."""
    rows = []
    for v in range(256):
        if fmt == "q6_k":
            h, t, l = v // 128, v % 128 // 32, v % 32
            rows.append((64 * h + 32 * (t % 2) + l, 4 * (t // 2), 128 + 32 * h + l, 2 * t, v // 16))
        else:
            c, h, i = v // 64, v % 64 // 32, v % 32
            at = 16 if fmt == "q4_k" else 48
            rows.append((at + 32 * c + i, 4 * h, 16 + i, 2 * c + h, v // 32))
    return torch.tensor(rows, device="cuda").T


def _values64(fmt, w):
    """f64 [rows, K], value by value from the formats' definition."""
    nbytes, values = BLOCK[fmt]
    b = w.reshape(w.shape[0], -1, nbytes)

    def half(at):
        return b[..., at:at + 2].clone().view(torch.float16).double()
    if fmt == "q8_0":
        return (half(0) * b[..., 2:].clone().view(torch.int8).double()).flatten(1)
    lo, ls, hi, hs, group = _table(fmt)
    q = (b[..., lo].int() >> ls.int()) & 15
    if fmt == "q6_k":
        q = q + 16 * ((b[..., hi].int() >> hs.int()) & 3) - 32
        return (q * b[..., 192:208].clone().view(torch.int8).double()[..., group] * half(208)).flatten(1)
    if fmt == "q5_k":
        q = q + 16 * ((b[..., hi].int() >> hs.int()) & 1)
    k = [[], []]
    for j in range(8):
        for which, at in ((0, 4), (1, 8)):
            if j < 4:
                k[which].append(b[..., at + j].int() & 63)
            else:
                k[which].append((b[..., 12 + j - 4].int() >> (4 * which)) % 16 + (b[..., at + j - 4].int() >> 6) * 16)
    sc, mn = (torch.stack(v, -1).double() for v in k)
    return (q * (half(0) * sc)[..., group] - (half(2) * mn)[..., group]).flatten(1)


def _act64(name, z):
    if name in ("none", "relu"):
        on = torch.ones_like(z) if name == "none" else torch.heaviside(z, torch.zeros_like(z))
        return z * on, on
    if name == "silu":
        s = torch.sigmoid(z)
        return z * s, s + z * s * torch.sigmoid(-z)
    if name == "gelu":
        s = torch.special.ndtr(z)
        return z * s, s + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)
    inner = math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3)
    slope = math.sqrt(2 / math.pi) * (1 + 3 * 0.044715 * z ** 2)
    return z / 2 * (1 + torch.tanh(inner)), (1 + torch.tanh(inner)) / 2 + z / 2 * slope / torch.cosh(inner.clamp(-300, 300)) ** 2


def exact(case, seed):
    """What run returns, in 64 bits from the definition (float64 on the GPU, a slab of weights at a time)."""
    s = prepare(case, seed)
    op, act, fmt, N, save = case["op"], case["act"], case["fmt"], case["N"], case["save"]
    slab = max(1, (1 << 25) // case["K"])
    if op.endswith("backward"):
        dy = s["grad"].double()
        pre = [p.double() for p in s["pre"]]
        if op == "gated_backward":
            a, da = _act64(act, pre[0])
            dz = [dy * pre[1] * da, dy * a]
        else:
            dz = [dy * _act64(act, pre[0])[1] if pre else dy]
        dx = torch.zeros((case["rows"], case["K"]), dtype=torch.float64, device="cuda")
        for d, w in zip(dz, s["weights"]):
            for i in range(0, N, slab):
                dx += d[:, i:i + slab] @ _values64(fmt, w[i:i + slab])
        return [dx] + (dz if save else [])
    x, z = s["x"].double(), []
    for w, b in zip(s["weights"], s["bias"]):
        p = torch.cat([x @ _values64(fmt, w[i:i + slab]).T for i in range(0, N, slab)], 1)
        z.append(p if b is None else p + b.double())
    y = _act64(act, z[0])[0]
    if op == "gated":
        y = y * z[1]
    elif s["residual"] is not None:
        y = y + s["residual"].double()
    return [y] + (z if save else [])
