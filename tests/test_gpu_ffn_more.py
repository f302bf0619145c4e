"""The feed-forward operators where their arithmetic is most at risk: rows of small f16 values, rows of one sign through blocks
whose minimum cancels their codes, activations far out on the way back, blocks of zeros behind large scales, weights that a
call shortly before has written.

Outputs are rounded to their type: an error of at most half a step, that of many values spread evenly over a step, whose
square is a twelfth of a step's on the average (`steps2`; of N values to within 1 / sqrt(N), for which a fifth more is given)."""
import numpy as np
import pytest
import torch

import ffn_ref
from test_gpu_ffn import ACT_ERR, DT, UNIT, Product, Weights, backward, check, clean, gated, mmq, project, rows

pytestmark = pytest.mark.gpu

MMQ_ERR_TIMEOUT = -7
BITS = {"f32": (24, -149), "bf16": (8, -133), "f16": (11, -24)}  # of a value, exponent of the smallest step


def steps2(want, dtype):
    """The square that roundings of `want` to its type add up to."""
    digits, least = BITS[dtype]
    e = torch.frexp(want)[1] - digits
    return float(torch.exp2(2.0 * e.clamp(min=least).double()).sum()) / 12 * 1.2


def pack(fmt, d, dmin, sc, mn, q):
    """Q4_K or Q5_K bytes [N, row bytes] of d, dmin [N, B], sc, mn [N, B, 8] and codes [N, B, 8, 32]."""
    N, B = d.shape
    out = np.zeros((N, B, ffn_ref.BYTES[fmt]), np.uint8)
    out[..., 0:2] = d.astype(np.float16)[..., None].view(np.uint8)
    out[..., 2:4] = dmin.astype(np.float16)[..., None].view(np.uint8)
    out[..., 4:8] = sc[..., :4] | sc[..., 4:] >> 4 << 6
    out[..., 8:12] = mn[..., :4] | mn[..., 4:] >> 4 << 6
    out[..., 12:16] = (sc[..., 4:] & 15) | (mn[..., 4:] & 15) << 4
    if fmt == "q5_k":
        for b in range(8):
            out[..., 16:48] |= (q[..., b, :] >> 4 & 1) << b
    low = (q & 15).reshape(N, B, 4, 2, 32)
    out[..., -128:] = (low[..., 0, :] | low[..., 1, :] << 4).reshape(N, B, 128)
    return out.reshape(N, -1)


class Blocks(Weights):
    """Normal weights as Q4_K or Q5_K: their minimum is half of the codes' range, as a quantizer leaves it."""

    def __init__(self, fmt, seed, N, K, by=0.02):
        rng = np.random.default_rng(seed)
        B, top = K // 256, 15 if fmt == "q4_k" else 31
        sc = rng.integers(35, 64, (N, B, 8)).astype(np.uint8)
        d = (rng.uniform(0.7, 1.3, (N, B)) * by * 4.6 / top / 50).astype(np.float16)
        dmin = (d.astype(np.float64) * (top / 2)).astype(np.float16)
        q = np.clip(np.rint(rng.standard_normal((N, B, 8, 32)) * (top / 4.6) + top / 2), 0, top).astype(np.uint8)
        raw = pack(fmt, d, dmin, sc, sc, q)
        v, size = ffn_ref.values(fmt, raw)
        self.fmt, self.N, self.K, self.bytes = fmt, N, K, torch.from_numpy(raw).cuda()
        self.v, self.size = torch.from_numpy(v).cuda(), torch.from_numpy(size).cuda()
        # of every 32-value block, and of every 256
        self.scale = torch.from_numpy((d.astype(np.float64)[..., None] * sc).reshape(N, -1)).cuda()
        self.dmin = torch.from_numpy(dmin.astype(np.float64)).cuda()


def block_sums(x, v):
    """sum over each block of 32 of x v: [M, N, K / 32] of x [M, K], v [N, K]."""
    return torch.einsum("mbk,nbk->mnb", x.view(x.shape[0], -1, 32), v.view(v.shape[0], -1, 32))


@pytest.mark.parametrize("fmt", ["q4_k", "q5_k"])
@pytest.mark.parametrize("M,N,K", [(1, 500, 1024), (16, 333, 512), (7, 200, 18944), (1, 150, 75776)])
@pytest.mark.parametrize("by", [1e-5, 1e-4, 1e-3, 1.0])
def test_few_f16_rows_of_any_size(fmt, M, N, K, by):
    """Up to 16 rows the codes enter exactly and rows to 2^-38 of their largest value.  What is left: a block's two products
    cut what lies 2^-24 below a product's exponent by its operands' fields, which a code as a subnormal has 2^10 too large: 34 cuts
    of 2^-14 of the block's largest x, and 17 of its sums in the minimum's product of a chunk."""
    w = Blocks(fmt, 3, N, K, by=1.0)
    x = rows(4, M, K, "f16", by)
    y = mmq.mmq_project(x, w.bytes, fmt, N)
    clean()
    xd = x.double()
    want = xd @ w.v.T
    top = xd.view(M, -1, 32).abs().amax(-1)
    sums = xd.view(M, -1, 8, 32).sum(-1).abs().amax(-1)
    cuts = (34 * 2.0 ** -14) ** 2 * top.square() @ w.scale.square().T + (17 * 2.0 ** -14) ** 2 * sums.square() @ w.dmin.square().T
    allowed = (float(cuts.sum()) + steps2(want, "f16")) ** 0.5
    off = float((y.double() - want).norm())
    assert off <= allowed, f"off by {off / float(want.norm()):.3g} of the norm, {allowed / float(want.norm()):.3g} is allowed"


@pytest.mark.parametrize("fmt", ["q4_k", "q5_k"])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("sign", ["any", "relu", "abs"])
@pytest.mark.parametrize("M,N,K", [(40, 300, 3584), (150, 257, 1024)])
def test_rows_of_one_sign_through_centred_blocks(fmt, dtype, sign, M, N, K):
    """A block's products with its codes and with its minimum are each many times their difference.  A weight is s (q - c) + r with
    c within 3/4 of minimum / s, so that nothing is as large as either: s off by 2^-11 (bf16 rows) of what its block
    comes to, r by 2^-11 of 3/4 s for all 32 alike, each weight by 2^-11 of itself; the tile's sum as everywhere."""
    w = Blocks(fmt, 5, N, K)
    x = rows(6, M, K, "f32")
    x = (x if sign == "any" else x.abs() if sign == "abs" else x.clamp(min=0)).to(DT[dtype])
    y = mmq.mmq_project(x, w.bytes, fmt, N)
    clean()
    xd = x.double()
    want = xd @ w.v.T
    most = 0.75 * xd.abs().view(M, -1, 32).sum(-1)[:, None] * w.scale[None]
    err = most if dtype == "f16" else 2 * most + block_sums(xd, w.v).abs()
    off2 = float(err.square().sum() + (xd.square() @ w.v.square().T).sum()) * 2.0 ** -22
    off2 += float(((K / 16 + 2) * 2.0 ** -22 * want).square().sum())
    allowed = (off2 + steps2(want, dtype)) ** 0.5
    off = float((y.double() - want).norm())
    assert off <= allowed, f"off by {off / float(want.norm()):.3g} of the norm, {allowed / float(want.norm()):.3g} is allowed"
    # and back: a row of gradients of one sign
    dy = xd[:, :N].to(DT[dtype])
    dx = mmq.mmq_project_backward(dy, w.bytes, fmt, K)
    clean()
    p = Product(dtype, [dy], [w], back=True)
    check(dx, p.z, p.err, p.walk, dtype, "dx")


@pytest.mark.parametrize("fmt", ["q4_k", "q5_k"])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_long_rows_of_one_sign_have_no_drift(fmt, dtype):
    """What weights are off by has no sign: over N output columns, whose weights are drawn apart, errors average out to their own size
    over sqrt(N), five of which are allowed (rows share their weights, so that all rows of a column count as one)."""
    M, N, K = 40, 500, 18944
    w = Blocks(fmt, 7, N, K)
    x = rows(8, M, K, "f32").abs().to(DT[dtype])
    y = mmq.mmq_project(x, w.bytes, fmt, N)
    clean()
    want = x.double() @ w.v.T
    off = (y.double() - want).mean(0)
    # a value's error: a part in 2^11 of its blocks' sums as above, some 2^-10 of the norm, and the outputs' rounding; f16's sums in the
    # tensor cores are cut towards zero, 2^-22 of them for every 16 values
    size = float((want.square().mean() * 2.0 ** -20 + steps2(want, dtype) / want.numel()).sqrt())
    cut = 2.0 ** -22 * K / 16 * float(want.abs().mean())
    assert abs(float(off.mean())) <= 5 * size / N ** 0.5 + cut, f"{float(off.mean()) / float(want.abs().mean()):.3g} of the mean size"


@pytest.mark.parametrize("act", [a for a in ffn_ref.ACTS if a != "none"])
@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
def test_derivatives_far_out(act, dtype):
    """Pre-activations of 10 to 1e20: the derivative is 0 or 1 to f32, and nothing overflows on the way."""
    N, K, far = 70, 64, [10.0, 100.0, 1e4] + ([1e10, 1e18, 1e20, 1e30] if dtype != "f16" else [6e4])
    z = torch.tensor([s * f for f in far for s in (1, -1)], device="cuda")
    M = z.numel()
    pre = (z[:, None] * (1 + torch.rand((M, N), device="cuda") / 16)).to(DT[dtype])
    up, dy = rows(1, M, N, dtype), rows(2, M, N, dtype)
    w = [Weights("q8_0", s, N, K) for s in (3, 4)]
    zd = pre.double()
    a, d = ffn_ref.act(act, zd.clamp(-60, 60))  # (beyond, the activation is z or 0 and its derivative 1 or 0, to e^-60)
    a, d = (torch.where(zd.abs() > 60, t, u) for t, u in ((zd.clamp(min=0), a), ((zd > 0).double(), d)))
    dz, dg, du = (torch.full((M, N), float("nan"), dtype=DT[dtype], device="cuda") for _ in range(3))
    dx = mmq.mmq_project_backward(dy, w[0].bytes, "q8_0", K, act=act, pre=pre, dz=dz)
    want = dy.double() * d
    err = ACT_ERR * 1.13 * dy.double().abs()
    check(dz, want, err, err, dtype, "dz")
    p = Product(dtype, [want], w[:1], back=True, formed=True)
    extra = err @ w[0].size
    check(dx, p.z, p.err + extra, p.walk + extra, dtype, "dx")
    small = up * 2.0 ** -10 if dtype == "f16" else up
    near = (a.abs() <= 1e4).all(1)  # (larger ones leave the other product's gradients far behind: their rows' own test is above)
    dx = mmq.mmq_gated_backward(small, pre, up, w[0].bytes, w[1].bytes, "q8_0", K, act=act, dgate=dg, dup=du)
    clean()
    sd = small.double()
    check(dg, sd * up.double() * d, ACT_ERR * 1.13 * (sd * up.double()).abs(), ACT_ERR * 1.13 * (sd * up.double()).abs(), dtype, "dg")
    check(du, sd * a, ACT_ERR * (sd * zd).abs(), ACT_ERR * (sd * zd).abs(), dtype, "du")
    assert torch.isfinite(dx).all()
    want = [sd * up.double() * d, sd * a]
    p = Product(dtype, [t[near] for t in want], w, back=True, formed=True)
    extra = ACT_ERR * 1.13 * ((sd * up.double()).abs()[near] @ w[0].size + (sd * zd).abs()[near] @ w[1].size)
    check(dx[near], p.z, p.err + extra, p.walk + extra, dtype, "dx")


@pytest.mark.parametrize("fmt", ["q4_k", "q5_k", "q6_k"])
@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
def test_blocks_of_zeros_behind_any_scale(fmt, dtype):
    """Sub-scales (and minimums) of 0 make zeros, whatever the block's scale: nothing there is out of range."""
    N, K, M = 130, 768, 40
    w = Weights(fmt, 3, N, K)
    raw = w.bytes.view(N, -1, ffn_ref.BYTES[fmt]).clone()
    at, zero = (208, slice(192, 208)) if fmt == "q6_k" else (0, slice(4, 16))
    raw[:, 1, zero] = 0
    out = []
    x, dy = rows(4, M, K, dtype), rows(5, M, N, dtype)
    for d in (0.0, 300.0, 65504.0):
        for i in (at,) if fmt == "q6_k" else (0, 2):
            raw[:, 1, i:i + 2] = torch.tensor(np.frombuffer(np.float16(d).tobytes(), np.uint8).copy(), device="cuda")
        b = raw.view(N, -1)
        out.append([mmq.mmq_project(x, b, fmt, N), mmq.mmq_project(x[:9], b, fmt, N), mmq.mmq_project_backward(dy, b, fmt, K)])
        clean()
    for other in out[1:]:
        assert all(torch.equal(a, b) for a, b in zip(out[0], other))


def test_weights_that_a_call_before_the_last_has_written():
    """The outputs of a long call are the weights of a short one, with another call between them: few rows, whose weights are
    asked for early, but never before the kernels up to the last but one have ended."""
    N, K = 512, 1 << 19
    long_w, x = torch.zeros((N, K // 32 * 34), dtype=torch.uint8, device="cuda"), rows(1, 1, K, "bf16")
    rng = np.random.default_rng(3)
    blocks = rng.integers(1, 100, (30, 34)).astype(np.uint8)  # (pairs of bytes that are finite bf16 values: a residual passes them on)
    blocks[:, 0:2] = np.frombuffer(np.float16(2.0 ** -7).tobytes(), np.uint8)
    wanted = torch.zeros(2 * N, dtype=torch.uint8)
    wanted[:blocks.size] = torch.from_numpy(blocks.reshape(-1))
    residual = wanted.view(torch.bfloat16).view(1, N).cuda()
    between, bx = Weights("q8_0", 2, 40, 64), rows(2, 3, 64, "bf16")
    cx = rows(3, 2, 32, "bf16")
    want = mmq.mmq_project(cx, wanted[:blocks.size].cuda(), "q8_0", 30)
    buf = torch.empty((1, N), dtype=torch.bfloat16, device="cuda")
    weights = buf.view(torch.uint8).view(-1)[:blocks.size]
    for _ in range(10):
        buf.zero_()
        torch.cuda.synchronize()
        mmq.mmq_project(x, long_w, "q8_0", N, residual=residual, out=buf)
        mmq.mmq_project(bx, between.bytes, "q8_0", 40)
        got = mmq.mmq_project(cx, weights, "q8_0", 30)
        torch.cuda.synchronize()
        assert torch.equal(buf, residual) and torch.equal(got, want)
    clean()


@pytest.mark.parametrize("fmt,dtype,call", [
    ("q4_k", "bf16", ("project", 40, 300, 9216)), ("q6_k", "f16", ("gated", 400, 9000, 256)), ("q5_k", "f32", ("project", 130, 520, 4096)),
    ("q8_0", "bf16", ("project", 70, 700, 288)), ("q4_k", "f32", ("back", 100, 4200, 512)), ("q6_k", "bf16", ("back", 300, 700, 2048)),
    ("q8_0", "f32", ("back", 33, 150, 288)), ("q4_k", "f16", ("back", 600, 300, 9216))])
def test_a_wait_that_gives_up_ends_the_call(fmt, dtype, call):
    """The wait for a unit's sums runs out, in all of the warps or in some: the call ends with a status, and the next one is right."""
    op, M, N, K = call
    w = [Weights(fmt, s, N, K).bytes for s in (1, 2)]
    x, dy = rows(3, M, K, dtype), rows(4, M, N, dtype)

    def run():
        if op == "back":
            return mmq.mmq_project_backward(dy, w[0], fmt, K)
        return mmq.mmq_gated(x, *w, fmt, N) if op == "gated" else mmq.mmq_project(x, w[0], fmt, N)
    want = run()
    clean()
    try:
        mmq.mmq_debug_set_wait_limit(0)  # (gives up where the sums are not there already, as some warps may find them)
        seen = set()
        for _ in range(40):
            run()
            torch.cuda.synchronize()
            seen.add(mmq.mmq_get_device_error())
        assert MMQ_ERR_TIMEOUT in seen and seen <= {0, MMQ_ERR_TIMEOUT}
    finally:
        mmq.mmq_debug_set_wait_limit(-1)
    assert torch.equal(run(), want)
    clean()


def weights_off(fmt, w, M):
    """What tiles make of the weights themselves, forward, less the weights: rows of the identity, M at a time, take them one
    by one, and a residual leaves of them what outputs in 16 bits would not show."""
    N, K = w.N, w.K
    out = {}
    for dtype in ("f16", "bf16"):
        near = w.v.T.contiguous().to(DT[dtype])
        eye = torch.eye(K, device="cuda", dtype=DT[dtype])
        y = torch.cat([mmq.mmq_project(eye[i:i + M], w.bytes, fmt, N, residual=-near[i:i + M]) for i in range(0, K, M)])
        clean()
        out[dtype] = (y.double() - (w.v.T - near.double())).T
        # (the outputs' rounding of what is left)
        out[dtype] = (out[dtype].abs() - (UNIT[dtype] * y.double().abs().T + (2.0 ** -25 if dtype == "f16" else 0.0))).clamp(min=0)
    return out


def close(fmt, w, off, scale, least):
    """Each weight within its bound: rounded once, 2^-11; what the minimum leaves of the nearest number of scales, `rest`, twice and its two
    parts before, 2^-11 each; for bf16 rows the scale's product with what is left of a code, 2^-11; numbers below f16's normal ones 2^-33."""
    size, rest, small = w.v.abs(), torch.zeros_like(w.v), 4 * 2.0 ** -33
    if least is not None:
        by = least / scale.clamp(min=1e-300)
        rest = torch.where(by <= 1000, (0.5 + by * 2.0 ** -9) * scale, least + 1000 * scale)
        rest = rest + 2.0 ** -10 * least
    for dtype, t in off.items():
        bound = 2.0 ** -11 * (size + 3 * rest + (size + rest if dtype == "bf16" and fmt != "q8_0" else 0)) * 1.01 + small
        worst = float((t / bound).max())
        assert worst <= 1.0, f"{dtype}: a weight is {worst:.3g} of its bound off"


@pytest.mark.parametrize("M", [32, 256])
@pytest.mark.parametrize("fmt", ["q4_k", "q5_k"])
@pytest.mark.parametrize("kind", ["any", "centred", "far", "sizes"])
def test_every_weight_with_a_minimum(fmt, kind, M):
    """Scales and minimums of either sign, of 0, far apart (a minimum of more than a thousand scales), from the smallest up to 250."""
    N, K = 72, 512
    rng = np.random.default_rng(4)
    B = K // 256
    sc, mn = (rng.integers(0, 64, (N, B, 8)).astype(np.uint8) for _ in range(2))
    q = rng.integers(0, 16 if fmt == "q4_k" else 32, (N, B, 8, 32)).astype(np.uint8)
    d, dmin = (rng.uniform(1e-4, 2e-3, (N, B)) * rng.choice([-1, 1], (N, B)) for _ in range(2))
    if kind == "centred":
        mn, dmin = sc, d * (7.5 if fmt == "q4_k" else 15.5)
    elif kind == "far":
        d = 2.0 ** rng.integers(-24, -8, (N, B)) * rng.choice([-1, 1], (N, B))
        dmin = np.clip(d * 2.0 ** rng.uniform(-6, 14, (N, B)), -3.9, 3.9)
    elif kind == "sizes":
        by = np.logspace(-5, np.log10(250), N)[:, None] / (63 * (32 if fmt == "q5_k" else 16) + 63)
        d, dmin = (by * rng.choice([-1, 1], (N, B)) for _ in range(2))
    d, dmin = (t.astype(np.float16) for t in (d, dmin))
    w = Weights.__new__(Weights)
    raw = pack(fmt, d, dmin, sc, mn, q)
    w.v, w.size = (torch.from_numpy(t).cuda() for t in ffn_ref.values(fmt, raw))
    w.fmt, w.N, w.K, w.bytes = fmt, N, K, torch.from_numpy(raw).cuda()
    scale, least = (torch.from_numpy(np.abs(t.astype(np.float64)[..., None] * u).reshape(N, -1).repeat(32, 1)).cuda()
                    for t, u in ((d, sc), (dmin, mn)))
    close(fmt, w, weights_off(fmt, w, M), scale, least)


@pytest.mark.parametrize("M", [32, 256])
@pytest.mark.parametrize("fmt", ["q6_k", "q8_0"])
@pytest.mark.parametrize("kind", ["any", "sizes"])
def test_every_weight_without_a_minimum(fmt, kind, M):
    N, K = 72, 512
    w = Weights(fmt, 3, N, K)
    if kind == "sizes":
        raw = w.bytes.cpu().numpy().reshape(N, -1, ffn_ref.BYTES[fmt]).copy()
        by = np.logspace(-5, np.log10(250), N)[:, None] / (128 * 32 if fmt == "q6_k" else 128)
        at = 208 if fmt == "q6_k" else 0
        raw[:, :, at:at + 2] = np.broadcast_to(by, raw.shape[:2]).astype(np.float16)[..., None].view(np.uint8)
        w.bytes = torch.from_numpy(raw.reshape(N, -1)).cuda()
        w.v = torch.from_numpy(ffn_ref.values(fmt, raw.reshape(N, -1))[0]).cuda()
    close(fmt, w, weights_off(fmt, w, M), None, None)


@pytest.mark.parametrize("fmt", ["q4_k", "q5_k", "q6_k", "q8_0"])
def test_f16_rows_report_weights_out_of_range(fmt):
    N, K, at = 150, 512, {"q6_k": 208}.get(fmt, 0)
    raw = Weights(fmt, 3, N, K).bytes.view(N, -1, ffn_ref.BYTES[fmt]).clone()
    x, dy, keep = rows(4, 40, K, "f16"), rows(5, 40, N, "f16"), [n for n in range(N) if n != 70]
    if fmt in ("q4_k", "q5_k"):
        raw[70, 1, 4:8] |= 16  # (sub-scales that are not all 0)
    good = mmq.mmq_project(x, raw.view(N, -1), fmt, N)
    clean()
    raw[70, 1, at:at + 2] = torch.tensor(np.frombuffer(np.float16(60000.0).tobytes(), np.uint8).copy(), device="cuda")
    bad = mmq.mmq_project(x, raw.view(N, -1), fmt, N)
    torch.cuda.synchronize()
    assert mmq.mmq_get_device_error() == -11
    assert torch.equal(good[:, keep], bad[:, keep])
    mmq.mmq_project_backward(dy, raw.view(N, -1), fmt, K)
    torch.cuda.synchronize()
    assert mmq.mmq_get_device_error() == -11


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("K", [128, 384, 640, 1152])
def test_q8_0_of_an_odd_number_of_128_values(dtype, K):
    """Rows off 16 bytes whose last chunk is a half: steps of 128 values, of which it has one."""
    for M, N in ((3, 40), (21, 131), (128, 300), (200, 70)):
        project("q8_0", dtype, M, N, K, seed=K)
        gated("q8_0", dtype, M, N, K, seed=K)
        backward("q8_0", dtype, M, N, K, 1, seed=K)
