"""The feed-forward operators on the GPU against their definition in 64 bits (tests/ffn_ref.py).

A product z = sum_k x_k w_k is off by at most, with size_k >= |w_k| the magnitudes that a weight is formed from
(code x scale, minimum) and S = sum |x_k| size_k:
  16-bit rows   weights in f16: scale, minimum and the weight itself rounded, 2^-11 each of at most size_k; a gradient
                that has been formed is rounded to f16 once more: 2^-11
  f32 rows      rows and weights in two f16 terms (2^-22 each), the product of the two small terms left out (2^-22)
                and the weight's own f32 value (2^-23)
  both          weights below f16's normal numbers, 2^-33 each (f16's half step 2^-25 below 2^-14, weights times 2^8), in
                each of the three roundings, and rows 2^-38 of their row's largest value in the same way
  sums          the tensor cores add 16 products to a running sum and round towards zero, 2^-22 of what is added:
                for f32 rows runs of 256 values, three products each, then f32 sums; else one run
That is the bound for each value (the largest error that can be).  Over many values the roundings of independent rows and
weights add up like a random walk: the whole output, as a vector, is off by at most sqrt(sum x_k^2 e_k^2) with e_k the
bound of weight k's error, beside the sums' part of the result's own size.
"""
import numpy as np
import pytest
import torch

import ffn_ref
import synth

mmq = pytest.importorskip("block_quantized_int8_mmq_gb300")
pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
UNIT = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8, "f16": 2.0 ** -11}
FMTS = ["q8_0", "q4_k", "q5_k", "q6_k"]
ACT_ERR = 2.0 ** -19  # activations in f32: arguments of exponentials up to 16, 2^-24 of them each, and a few roundings


def clean():
    torch.cuda.synchronize()
    assert mmq.mmq_get_device_error() == 0


class Weights:
    def __init__(self, fmt, seed, N, K):
        w = synth.weights(fmt, seed, N, K)
        v, size = ffn_ref.values(fmt, w)
        self.fmt, self.N, self.K, self.bytes = fmt, N, K, torch.from_numpy(w).cuda()
        self.v, self.size = torch.from_numpy(v).cuda(), torch.from_numpy(size).cuda()


def rows(seed, M, N, dtype, by=1.0):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn((M, N), device="cuda", generator=gen) * by).to(DT[dtype])


class Product:
    """x W^T (or x W) in 64 bits with its bounds: z, each value's largest error, and the whole's as a walk."""

    def __init__(self, dtype, x, ws, back=False, formed=False):
        xs = [t.double() for t in x]
        wide = dtype == "f32"
        self.z = self.err = self.walk = 0
        for t, w in zip(xs, ws):
            v, size = (w.v, w.size) if back else (w.v.T, w.size.T)
            if wide:
                e, ex = 2.0 ** -22 * size + 2.0 ** -23 * size + 2.0 ** -33, 2.0 ** -21
            else:
                e, ex = 2.0 ** -10 * 1.01 * size + 3 * 2.0 ** -33, 2.0 ** -11 if formed else 0.0
            top = t.abs().amax(1, keepdim=True) if t.shape[1] else t.abs()
            K = v.shape[0]
            sums = (2.0 ** -22 * (50 + K / 256) if wide else 2.0 ** -22 * (K / 16 + 2))
            self.z = self.z + t @ v
            S = t.abs() @ size
            self.err = self.err + t.abs() @ e + (ex + sums) * S + 2.0 ** -38 * top * size.sum(0)
            self.walk = self.walk + t.square() @ e.square() + ex * ex * (t.square() @ size.square())
        self.walk = (self.walk.sqrt() * 1.1 + sums * self.z.abs() + 2.0 ** -38 * top * size.sum(0))


def check(got, want, err, walk, dtype, what=""):
    """got within err of want value by value, and within walk as a whole, beside the rounding to its type."""
    assert got.shape == want.shape
    g = got.double()
    assert torch.isfinite(g).all(), what
    u = UNIT[dtype]
    floor = 2.0 ** -25 if dtype == "f16" else 0.0
    bound = err + u * (want.abs() + err) + floor
    off = (g - want).abs()
    worst = float((off / bound.clamp(min=1e-300)).max())
    assert worst <= 1.0, f"{what}: a value is {worst:.3g} of its bound off"
    total = float(((walk + u * want.abs() + floor).square().sum()).sqrt())
    assert float(off.norm()) <= total, f"{what}: off by {float(off.norm()):.3g}, {total:.3g} is allowed"


def epilogue(dtype, act, parts):
    """act(z0) * z1 (or act(z0) alone) with the bounds carried through: |act'| <= 1.13."""
    a, _ = ffn_ref.act(act, parts[0][0])
    out = []
    for i in (1, 2):
        d = 1.13 * parts[0][i] + ACT_ERR * a.abs()
        if len(parts) == 2:
            d = d * (parts[1][0].abs() + parts[1][i]) + a.abs() * parts[1][i]
        out.append(d)
    return (a * parts[1][0] if len(parts) == 2 else a), out[0], out[1]


def biased(p, b):
    z = p.z if b is None else p.z + b.double()
    return z, p.err + 2.0 ** -23 * z.abs(), p.walk + 2.0 ** -23 * z.abs()


def project(fmt, dtype, M, N, K, act=None, bias=False, residual=False, pre=False, seed=1, x=None, by=1.0):
    w = Weights(fmt, seed, N, K)
    x = rows(seed + 1, M, K, dtype, by) if x is None else x
    b = torch.randn((N,), device="cuda") if bias else None
    r = rows(seed + 2, M, N, dtype) if residual else None
    kept = torch.full((M, N), float("nan"), dtype=DT[dtype], device="cuda") if pre else None
    y = mmq.mmq_project(x, w.bytes, fmt, N, bias=b, act=act, residual=r, pre=kept)
    clean()
    z = biased(Product(dtype, [x], [w]), b)
    a, err, walk = epilogue(dtype, act or "none", [z])
    if residual:
        a = a + r.double()
        err, walk = err + 2.0 ** -24 * a.abs(), walk + 2.0 ** -24 * a.abs()
    check(y, a, err, walk, dtype, "y")
    if pre:
        check(kept, *z, dtype, "pre")
    return x, w, y


def gated(fmt, dtype, M, N, K, act="silu", bias=False, keep=False, seed=1, by=1.0):
    w = [Weights(fmt, seed + i, N, K) for i in (0, 100)]
    x = rows(seed + 1, M, K, dtype, by)
    b = [torch.randn((N,), device="cuda") if bias else None for _ in w]
    kept = [torch.full((M, N), float("nan"), dtype=DT[dtype], device="cuda") if keep else None for _ in w]
    h = mmq.mmq_gated(x, w[0].bytes, w[1].bytes, fmt, N, act=act, bias_gate=b[0], bias_up=b[1], gate=kept[0], up=kept[1])
    clean()
    z = [biased(Product(dtype, [x], [wi]), bi) for wi, bi in zip(w, b)]
    check(h, *epilogue(dtype, act, z), dtype, "h")
    if keep:
        check(kept[0], *z[0], dtype, "gate")
        check(kept[1], *z[1], dtype, "up")


def formed(dtype, dy, act, pre):
    """dz in 64 bits and whether the rows of the product have been rounded once more."""
    a, d = ffn_ref.act(act, pre[0].double()) if pre else (None, torch.ones(()).cuda().double())
    dz = [dy.double() * d]
    if pre and len(pre) == 2:
        dz = [dz[0] * pre[1].double(), dy.double() * a]
    return dz


def backward(fmt, dtype, M, N, K, mats, act="silu", keep=False, seed=1, fall=True):
    w = [Weights(fmt, seed + 100 * i, N, K) for i in range(mats)]
    dy = rows(seed + 1, M, N, dtype)
    if fall:  # rows of very different sizes
        dy = (dy.float() * torch.logspace(0, -4, M, device="cuda")[:, None]).to(DT[dtype])
    pre = [rows(seed + 2 + i, M, N, dtype, 1.5) for i in range(mats)] if mats == 2 or act != "none" else []
    kept = [torch.full((M, N), float("nan"), dtype=DT[dtype], device="cuda") if keep else None for _ in w]
    if mats == 2:
        dx = mmq.mmq_gated_backward(dy, pre[0], pre[1], w[0].bytes, w[1].bytes, fmt, K, act=act, dgate=kept[0], dup=kept[1])
    else:
        dx = mmq.mmq_project_backward(dy, w[0].bytes, fmt, K, act=act, pre=pre[0] if pre else None, dz=kept[0])
    clean()
    dz = formed(dtype, dy, act, pre)
    p = Product(dtype, dz, w, back=True, formed=True)
    # the gradients themselves, formed in f32: factors of up to 1.13 |dy u| that may nearly cancel
    size = [1.13 * dy.double().abs() * (pre[1].double().abs() if mats == 2 else 1.0), dy.double().abs() *
            (pre[0].double().abs() if mats == 2 else 1.0)]
    extra = sum(ACT_ERR * size[i] @ w[i].size for i in range(mats))
    check(dx, p.z, p.err + extra, p.walk + extra, dtype, "dx")
    for i in range(mats):
        if keep:
            check(kept[i], dz[i], ACT_ERR * size[i], ACT_ERR * size[i], dtype, f"dz {i}")


# ------------------------------------------------------------------------------------------ sizes
@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("M,N,K", [(1, 1, 256), (3, 130, 512), (8, 256, 768), (17, 127, 256), (65, 300, 1280), (200, 257, 512),
                                   (129, 513, 2304)])
def test_project_sizes(fmt, dtype, M, N, K):
    project(fmt, dtype, M, N, K)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("M,N,K", [(1, 5, 512), (2, 129, 256), (9, 200, 1024), (33, 128, 768), (97, 385, 512), (193, 140, 256)])
def test_gated_sizes(fmt, dtype, M, N, K):
    gated(fmt, dtype, M, N, K, keep=M % 2 == 1)


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("K", [32, 64, 96, 224, 288, 544, 1056])
def test_q8_0_of_any_number_of_blocks(dtype, K):
    """Rows of 34 K / 32 bytes: every alignment to 16, steps of 64 values that the last block does not fill."""
    for M, N in ((1, 40), (21, 131)):
        project("q8_0", dtype, M, N, K, seed=K)
        gated("q8_0", dtype, M, N, K, seed=K)
        backward("q8_0", dtype, M, N, K, 2, seed=K)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("M,N,K", [(1, 1, 256), (2, 33, 512), (8, 64, 256), (19, 65, 768), (66, 127, 1280), (194, 320, 512),
                                   (40, 1000, 256)])
def test_backward_sizes(fmt, dtype, M, N, K):
    backward(fmt, dtype, M, N, K, 1, act="none", seed=3)
    backward(fmt, dtype, M, N, K, 2, keep=M % 2 == 0, seed=5)


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("M", [1, 7, 8, 15, 16, 24, 47, 63, 64, 66, 95, 96, 128, 160, 191, 192, 208, 385, 577])
def test_every_tile_of_rows(dtype, M):
    project("q4_k", dtype, M, 150, 512, seed=M)
    backward("q5_k", dtype, M, 70, 512, 1, act="none", seed=M)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("M", [1, 20, 250])
def test_long_sums_shared_out(fmt, dtype, M):
    """Few tiles of outputs, long sums: the work on one output is shared by several workers."""
    project(fmt, dtype, M, 200, 9216, residual=True, seed=2)
    backward(fmt, dtype, M, 4200, 256, 1, act="relu", seed=2)


@pytest.mark.parametrize("fmt,dtype", [("q4_k", "bf16"), ("q6_k", "f32"), ("q8_0", "f16")])
def test_more_tiles_than_workers(fmt, dtype):
    gated(fmt, dtype, 400, 9000, 256, seed=4)
    project(fmt, dtype, 700, 8200, 512, seed=4)
    backward(fmt, dtype, 600, 300, 9216, 2, seed=4)


# --------------------------------------------------------------------------------------- epilogues
@pytest.mark.parametrize("act", ffn_ref.ACTS)
@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("M", [3, 70])
def test_epilogues(act, dtype, M):
    for bias in (False, True):
        for residual in (False, True):
            project("q5_k", dtype, M, 140, 512, act=act, bias=bias, residual=residual, pre=bias != residual, seed=7)
        gated("q8_0", dtype, M, 140, 512, act=act, bias=bias, keep=bias, seed=8)
    backward("q4_k", dtype, M, 140, 512, 1, act=act, keep=True, seed=9)
    backward("q6_k", dtype, M, 140, 512, 2, act=act, keep=True, seed=9)


@pytest.mark.parametrize("act", ffn_ref.ACTS)
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_activations_far_out(act, dtype):
    """Pre-activations of up to some hundreds: exponentials run out of range on both sides."""
    project("q8_0", dtype, 40, 64, 256, act=act, seed=3, by=400.0)
    gated("q8_0", dtype, 40, 64, 256, act=act, seed=3, by=400.0)


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
def test_rows_of_every_size(dtype):
    """Rows from the type's smallest to large ones; a row of zeros; one value far above the others."""
    M = 40
    by = torch.logspace(-4, 1, M, device="cuda") if dtype == "f16" else torch.logspace(-30, 12, M, device="cuda")
    x = (rows(5, M, 512, "f32") * by[:, None]).to(DT[dtype])
    x[3] = 0
    x[7, 100] = 1e4 * float(by[7])
    project("q6_k", dtype, M, 130, 512, seed=6, x=x)
    backward("q6_k", dtype, M, 130, 512, 1, act="none", seed=6)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_weights_of_every_size(fmt, dtype):
    """Scales from far below f16's normal numbers up to weights of 200."""
    N, K = 96, 512
    w = Weights(fmt, 3, N, K)
    raw = synth.weights(fmt, 3, N, K).reshape(N, -1, ffn_ref.BYTES[fmt])
    top = np.abs(w.size.cpu().numpy()).max(1)
    f = np.logspace(np.log10(1e-4), np.log10(0.9 * 200), N) / top
    for at in {"q8_0": (0,), "q6_k": (208,)}.get(fmt, (0, 2)):
        d = raw[:, :, at:at + 2].copy().view(np.float16).astype(np.float64) * f[:, None, None]
        raw[:, :, at:at + 2] = d.astype(np.float16).view(np.uint8).reshape(N, -1, 2)
    w.bytes = torch.from_numpy(raw.reshape(N, -1)).cuda()
    w.v, w.size = (torch.from_numpy(t).cuda() for t in ffn_ref.values(fmt, raw.reshape(N, -1)))
    for M in (1, 50):
        x = rows(4, M, K, dtype)
        y = mmq.mmq_project(x, w.bytes, fmt, N)
        p = Product(dtype, [x], [w])
        check(y, p.z, p.err, p.walk, dtype, "y")
        dy = rows(5, M, N, dtype)
        dx = mmq.mmq_project_backward(dy, w.bytes, fmt, K)
        p = Product(dtype, [dy], [w], back=True)
        check(dx, p.z, p.err, p.walk, dtype, "dx")
    clean()


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("M", [5, 120])
def test_what_is_not_finite_stays_in_its_row(dtype, M):
    N, K = 140, 512
    w = Weights("q4_k", 1, N, K)
    x, dy = rows(1, M, K, dtype), rows(2, M, N, dtype)
    good = [mmq.mmq_project(x, w.bytes, "q4_k", N, act="relu"), mmq.mmq_gated(x, w.bytes, w.bytes, "q4_k", N),
            mmq.mmq_project_backward(dy, w.bytes, "q4_k", K)]
    x[1, 7], x[3, 300], dy[1, 9], dy[3, 100] = float("nan"), float("inf"), float("nan"), float("-inf")
    bad = [mmq.mmq_project(x, w.bytes, "q4_k", N, act="relu"), mmq.mmq_gated(x, w.bytes, w.bytes, "q4_k", N),
           mmq.mmq_project_backward(dy, w.bytes, "q4_k", K)]
    clean()
    keep = [i for i in range(M) if i not in (1, 3)]
    for g, b in zip(good, bad):
        assert torch.equal(g[keep], b[keep])
        assert not torch.isfinite(b[1]).any() and not torch.isfinite(b[3]).all()


# ------------------------------------------------------------------------------- strides and places
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("M", [4, 100])
def test_strided_rows_and_a_residual_in_place(dtype, M):
    N, K = 141, 512
    w = Weights("q6_k", 2, N, K)
    wide = rows(3, M, 3 * K, dtype)
    x = wide[:, K:2 * K]
    r = rows(4, M, N + 11, dtype)[:, 5:5 + N]  # rows aligned to their elements only
    a = mmq.mmq_project(x, w.bytes, "q6_k", N, residual=r)
    assert torch.equal(a, mmq.mmq_project(x.contiguous(), w.bytes, "q6_k", N, residual=r.contiguous()))
    out = r.contiguous().clone()
    assert torch.equal(mmq.mmq_project(x, w.bytes, "q6_k", N, residual=out, out=out), a)
    g = mmq.mmq_gated(x, w.bytes, w.bytes, "q6_k", N)
    assert torch.equal(g, mmq.mmq_gated(x.contiguous(), w.bytes, w.bytes, "q6_k", N))
    dy = rows(5, M, N + 7, dtype)[:, 3:3 + N]
    d = mmq.mmq_project_backward(dy, w.bytes, "q6_k", K)
    assert torch.equal(d, mmq.mmq_project_backward(dy.contiguous(), w.bytes, "q6_k", K))
    d = mmq.mmq_gated_backward(dy, a, g, w.bytes, w.bytes, "q6_k", K)
    assert torch.equal(d, mmq.mmq_gated_backward(dy.contiguous(), a, g, w.bytes, w.bytes, "q6_k", K))
    clean()


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("M", [3, 77])
def test_nothing_beside_the_outputs_is_written(fmt, M):
    N, K = 139, 768
    w, guard = Weights(fmt, 2, N, K), 4096

    def place(n):
        whole = torch.full((guard + n + guard,), 7.0, dtype=torch.bfloat16, device="cuda")
        return whole, whole[guard:guard + n]
    for args in ((M, N), (M, K)):
        whole, mid = place(args[0] * args[1])
        more, kept = place(M * N)
        if args[1] == N:
            mmq.mmq_project(rows(1, M, K, "bf16"), w.bytes, fmt, N, pre=kept.view(M, N), out=mid.view(M, N))
            assert torch.equal(kept, mid)
        else:
            dy = rows(1, M, N, "bf16")
            mmq.mmq_project_backward(dy, w.bytes, fmt, K, dz=kept.view(M, N), dx=mid.view(M, K))
            assert torch.equal(kept.view(M, N), dy)
        clean()
        for t in (whole, more):
            assert bool((t[:guard] == 7).all()) and bool((t[-guard:] == 7).all())


def test_weights_that_end_where_their_memory_does():
    """Rows of 210 bytes and of 34: copies of whole 16 bytes must not run past the last row."""
    for fmt, K, N in (("q6_k", 256, 5), ("q8_0", 32, 3), ("q8_0", 96, 7), ("q6_k", 768, 129)):
        w = Weights(fmt, 9, N, K)
        size = w.bytes.numel()
        whole = torch.full((size + 64,), 255, dtype=torch.uint8, device="cuda")
        whole[:size] = w.bytes.view(-1)
        x, dy = rows(1, 6, K, "f16"), rows(2, 6, N, "f16")
        a, d = mmq.mmq_project(x, w.bytes, fmt, N), mmq.mmq_project_backward(dy, w.bytes, fmt, K)
        view = whole[:size].view(N, -1)
        assert torch.equal(a, mmq.mmq_project(x, view, fmt, N))
        assert torch.equal(d, mmq.mmq_project_backward(dy, view, fmt, K))
    clean()


def test_more_than_2_31_outputs():
    """Offsets past 32 bits in the outputs and in the rows."""
    M, N, K = 120000, 18944, 256
    if torch.cuda.mem_get_info()[0] < 40 << 30:
        pytest.skip("needs 40 GB")
    w = Weights("q4_k", 2, N, K)
    x = rows(1, M, K, "bf16")
    y = mmq.mmq_project(x, w.bytes, "q4_k", N)
    pick = torch.tensor([0, 1, 59999, 113359, 113360, 119998, 119999], device="cuda")
    p = Product("bf16", [x[pick]], [w])
    check(y[pick], p.z, p.err, p.walk, "bf16", "y")
    dx = mmq.mmq_project_backward(y, w.bytes, "q4_k", K)
    p = Product("bf16", [y[pick]], [w], back=True)
    check(dx[pick], p.z, p.err, p.walk, "bf16", "dx")
    clean()


def test_no_rows():
    w = Weights("q4_k", 1, 20, 256)
    for dtype in DT:
        x, g = rows(1, 0, 256, dtype), rows(1, 0, 20, dtype)
        assert mmq.mmq_project(x, w.bytes, "q4_k", 20).shape == (0, 20)
        assert mmq.mmq_gated(x, w.bytes, w.bytes, "q4_k", 20).shape == (0, 20)
        assert mmq.mmq_project_backward(g, w.bytes, "q4_k", 256).shape == (0, 256)
        assert mmq.mmq_gated_backward(g, g, g, w.bytes, w.bytes, "q4_k", 256).shape == (0, 256)
    clean()


# ------------------------------------------------------------------------ gradients, streams, graphs
@pytest.mark.parametrize("fmt,act", [("q4_k", "silu"), ("q6_k", "gelu"), ("q8_0", "gelu_tanh"), ("q5_k", "none")])
def test_gradients_against_differences(fmt, act):
    """d/dt of sum(c * h(x + t v)) at 0 by central differences of the f32 forward pass, t = 2^-7: the
    differences' own error is t^2 / 6 times a third derivative of order one for pre-activations of order one, and f32
    rounding over t; both below 2^-10 of the terms' sizes."""
    M, N, K, t = 6, 96, 512, 2.0 ** -7
    w = [Weights(fmt, s, N, K) for s in (1, 2)]
    by = 1.0 / float((w[0].v.square().sum(1)).mean().sqrt())
    x, v, c = rows(1, M, K, "f32", by), rows(2, M, K, "f32", by), rows(3, M, N, "f32")

    def h(at):
        return mmq.mmq_gated(at, w[0].bytes, w[1].bytes, fmt, N, act=act).double()
    gate, up = (torch.empty((M, N), device="cuda") for _ in range(2))
    mmq.mmq_gated(x, w[0].bytes, w[1].bytes, fmt, N, act=act, gate=gate, up=up)
    dx = mmq.mmq_gated_backward(c, gate, up, w[0].bytes, w[1].bytes, fmt, K, act=act)
    want = (c.double() * (h(x + t * v) - h(x - t * v))).sum(1) / (2 * t)
    got = (dx.double() * v.double()).sum(1)
    assert float((got - want).abs().max()) <= 2.0 ** -10 * float((c.double().abs() * 2).sum(1).max())

    def y(at):
        return mmq.mmq_project(at, w[0].bytes, fmt, N, act=act).double()
    mmq.mmq_project(x, w[0].bytes, fmt, N, act=act, pre=gate)
    dx = mmq.mmq_project_backward(c, w[0].bytes, fmt, K, act=act, pre=gate)
    want = (c.double() * (y(x + t * v) - y(x - t * v))).sum(1) / (2 * t)
    got = (dx.double() * v.double()).sum(1)
    assert float((got - want).abs().max()) <= 2.0 ** -10 * float((c.double().abs() * 2).sum(1).max())
    clean()


def block(x, w, dtype):
    """The feed-forward block forward and back, as a training step over frozen weights runs it."""
    M, K = x.shape
    N = w[0].N
    gate, up = (torch.empty((M, N), dtype=x.dtype, device="cuda") for _ in range(2))
    h = mmq.mmq_gated(x, w[0].bytes, w[1].bytes, "q4_k", N, gate=gate, up=up)
    y = mmq.mmq_project(h, w[2].bytes, "q6_k", K, residual=x)
    dh = mmq.mmq_project_backward(y, w[2].bytes, "q6_k", N)
    dx = mmq.mmq_gated_backward(dh, gate, up, w[0].bytes, w[1].bytes, "q4_k", K)
    return y, dx


@pytest.mark.parametrize("dtype,M", [("f32", 1), ("f32", 90), ("bf16", 1), ("bf16", 200), ("f16", 37)])
def test_a_block_forward_and_back(dtype, M):
    """The four operators one after another.  Each one's inputs are what the one before gave, so each is held
    to its own bounds by the tests above; here the whole is, to the roundings of its stages: 8 of the type's half steps
    and of the weights' (16-bit rows: 2^-10) of the vectors' sizes."""
    N, K = 512, 768
    w = [Weights("q4_k", 1, N, K), Weights("q4_k", 2, N, K), Weights("q6_k", 3, K, N)]
    x = rows(4, M, K, dtype, 0.02)
    y, dx = block(x, w, dtype)
    clean()
    xd = x.double()
    g, u = xd @ w[0].v.T, xd @ w[1].v.T
    a, d = ffn_ref.act("silu", g)
    want = (a * u) @ w[2].v.T + xd
    dh = y.double() @ w[2].v
    want_dx = (dh * u * d) @ w[0].v + (dh * a) @ w[1].v
    tol = 8 * (UNIT[dtype] + (2.0 ** -10 if dtype != "f32" else 2.0 ** -17))
    assert float((y.double() - want).norm()) <= tol * float(want.norm())
    assert float((dx.double() - want_dx).norm()) <= 2 * tol * float(want_dx.norm())


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("M", [1, 70])
def test_repeated_calls_give_the_same_bits(dtype, M):
    w = Weights("q5_k", 1, 300, 4096)
    x, dy = rows(1, M, 4096, dtype), rows(2, M, 300, dtype)
    a, d = mmq.mmq_project(x, w.bytes, "q5_k", 300), mmq.mmq_project_backward(dy, w.bytes, "q5_k", 4096)
    for _ in range(10):
        assert torch.equal(a, mmq.mmq_project(x, w.bytes, "q5_k", 300))
        assert torch.equal(d, mmq.mmq_project_backward(dy, w.bytes, "q5_k", 4096))


@pytest.mark.parametrize("M", [1, 40])
def test_two_captured_graphs_side_by_side(M):
    """Two graphs of the same calls on two streams at once, replayed with changed rows: nothing of one is the other's."""
    w = [Weights("q4_k", 1, 512, 768), Weights("q4_k", 2, 512, 768), Weights("q6_k", 3, 768, 512)]
    xs = [rows(5 + i, M, 768, "bf16", 0.02) for i in range(2)]
    block(xs[0], w, "bf16")
    torch.cuda.synchronize()
    graphs, outs, streams = [], [], [torch.cuda.Stream() for _ in range(2)]
    for x in xs:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(block(x, w, "bf16"))
        graphs.append(g)
    for trip in range(5):
        for i, x in enumerate(xs):
            x.copy_(rows(50 + 2 * trip + i, M, 768, "bf16", 0.02))
        torch.cuda.synchronize()
        for _ in range(3):
            for g, s in zip(graphs, streams):
                with torch.cuda.stream(s):
                    g.replay()
        torch.cuda.synchronize()
        for x, o in zip(xs, outs):
            for a, b in zip(o, block(x, w, "bf16")):
                assert torch.equal(a, b)
    clean()


@pytest.mark.parametrize("raw", [False, True])
def test_two_streams_at_once(raw):
    w = [Weights("q4_k", 1, 512, 768), Weights("q4_k", 2, 512, 768)]
    x = [rows(5 + i, 60, 768, "bf16", 0.02) for i in range(4)]
    want = [mmq.mmq_gated(t, w[0].bytes, w[1].bytes, "q4_k", 512) for t in x]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in x]
    for _ in range(20):
        got = [mmq.mmq_gated(t, w[0].bytes, w[1].bytes, "q4_k", 512, stream=s.cuda_stream if raw else s)
               for t, s in zip(x, streams)]
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a, b)
    clean()


def test_a_chain_without_a_pause():
    """Calls that follow one another read what the one before wrote, and reuse its scratch memory."""
    w = Weights("q6_k", 3, 512, 512)
    x = rows(1, 33, 512, "f16")
    steps = [x]
    for _ in range(30):
        y = mmq.mmq_project(steps[-1], w.bytes, "q6_k", 512, act="relu")
        steps.append((y / 64))
    torch.cuda.synchronize()
    for a, b in zip(steps, steps[1:]):
        assert torch.equal(mmq.mmq_project(a, w.bytes, "q6_k", 512, act="relu") / 64, b)
    a = mmq.mmq_project(x, w.bytes, "q6_k", 512, act="relu")
    torch.cuda.synchronize()
    for _ in range(20):
        b = mmq.mmq_project(mmq.mmq_project(x, w.bytes, "q6_k", 512, act="relu"), w.bytes, "q6_k", 512)
        assert torch.equal(b, mmq.mmq_project(a, w.bytes, "q6_k", 512))
    clean()


# ---------------------------------------------------------------------------------------- refusals
def test_python_refusals():
    N, K = 20, 256
    w = Weights("q4_k", 1, N, K).bytes
    x, dy = rows(1, 3, K, "bf16"), rows(2, 3, N, "bf16")
    bias = torch.zeros((N,), device="cuda")
    bad = [dict(x=x.double()), dict(x=x[0]), dict(x=x.T), dict(wq=w[:-1]), dict(wq=w.cpu()), dict(wq=w.view(torch.int8)),
           dict(fmt="q3_k"), dict(fmt=None), dict(N=N + 1), dict(act="tanh"), dict(bias=bias.double()), dict(bias=bias[:-1]),
           dict(residual=x), dict(residual=dy.float()), dict(pre=dy.float()), dict(pre=dy.T), dict(out=dy[:2]),
           dict(out=rows(1, 3, 2 * N, "bf16")[:, :N])]
    for change in bad:
        a = dict(x=x, wq=w, fmt="q4_k", N=N)
        a.update(change)
        with pytest.raises(ValueError):
            mmq.mmq_project(**a)
    for change in (dict(w_up=w[1:]), dict(gate=x), dict(up=dy.float()), dict(bias_up=bias[1:]), dict(act=7), dict(x=x.cpu())):
        a = dict(x=x, w_gate=w, w_up=w, fmt="q4_k", N=N)
        a.update(change)
        with pytest.raises(ValueError):
            mmq.mmq_gated(**a)
    for change in (dict(dy=x), dict(K=2 * K), dict(pre=x), dict(dz=x), dict(dx=dy)):
        a = dict(dy=dy, wq=w, fmt="q4_k", K=K, act="silu", pre=dy)
        a.update(change)
        with pytest.raises(ValueError):
            mmq.mmq_project_backward(**a)
    with pytest.raises(mmq.MMQError):
        mmq.mmq_project_backward(dy, w, "q4_k", K, act="silu")  # an activation without its pre-activations
    for change in (dict(gate=x), dict(up=dy.float()), dict(dgate=x), dict(dup=dy[:1]), dict(w_gate=w[1:])):
        a = dict(dh=dy, gate=dy, up=dy, w_gate=w, w_up=w, fmt="q4_k", K=K)
        a.update(change)
        with pytest.raises(ValueError):
            mmq.mmq_gated_backward(**a)
    # a row that does not begin on 16 bytes
    with pytest.raises(mmq.MMQError):
        mmq.mmq_project(rows(1, 3, K + 8, "bf16")[:, 4:4 + K], w, "q4_k", N)
    clean()


@pytest.mark.parametrize("M", [3, 40])
def test_a_refused_call_writes_nothing(M, capfd):
    """Shared memory that is refused: MMQ_ERR_SMEM before anything is launched, the gradients' outputs included."""
    N, K = 4200, 256
    w = Weights("q4_k", 1, 20, K)
    wide = torch.zeros((N, K // 256 * 144), dtype=torch.uint8, device="cuda")
    x, dy = rows(1, M, K, "f32"), rows(2, M, N, "f32")
    out, dz, dx = (torch.full(s, 7.0, device="cuda") for s in ((M, 20), (M, N), (M, K)))
    mmq.mmq_debug_refuse_smem(True)
    try:
        for call in (lambda: mmq.mmq_project(x, w.bytes, "q4_k", 20, out=out),
                     lambda: mmq.mmq_project_backward(dy, wide, "q4_k", K, act="relu", pre=dy, dz=dz, dx=dx)):
            with pytest.raises(mmq.MMQError) as e:
                call()
            assert e.value.status == -5
    finally:
        mmq.mmq_debug_refuse_smem(False)
    clean()
    assert all(bool((t == 7).all()) for t in (out, dz, dx))
    assert "refused" in capfd.readouterr().err


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_weights_out_of_range_are_reported(fmt, dtype):
    """Magnitudes past 255: the error word says so; other columns keep their values.  Up to 16 rows take any weights."""
    N, K, at = 150, 512, {"q6_k": 208}.get(fmt, 0)
    w = Weights(fmt, 3, N, K)
    raw = w.bytes.view(N, -1, ffn_ref.BYTES[fmt]).clone()
    raw[70, 1, at:at + 2] = torch.tensor(np.frombuffer(np.float16(60000.0).tobytes(), np.uint8).copy(), device="cuda")
    if fmt in ("q4_k", "q5_k"):
        raw[70, 1, 4:8] |= 16  # (sub-scales that are not all 0)
    raw = raw.view(N, -1)
    x, keep = rows(4, 40, K, dtype), [n for n in range(N) if n != 70]
    good = mmq.mmq_project(x, w.bytes, fmt, N)
    clean()
    bad = mmq.mmq_project(x, raw, fmt, N)
    torch.cuda.synchronize()
    assert mmq.mmq_get_device_error() == -11
    assert torch.equal(good[:, keep], bad[:, keep])
    dy = rows(5, 40, N, dtype)
    mmq.mmq_project_backward(dy, raw, fmt, K)
    torch.cuda.synchronize()
    assert mmq.mmq_get_device_error() == -11
    big = ffn_ref.values(fmt, raw.cpu().numpy())
    if dtype == "f32":
        few = mmq.mmq_project(x[:5], raw, fmt, N)
        clean()
        want = x[:5].double() @ torch.from_numpy(big[0]).cuda().T
        size = x[:5].double().abs() @ torch.from_numpy(big[1]).cuda().T
        assert bool(((few.double() - want).abs() <= 2.0 ** -16 * size).all())


@pytest.mark.parametrize("M", [2, 16, 17, 130])
def test_a_first_call_inside_a_capture(M):
    """Nothing has to run before a capture: in a process of its own, the first call of each operator is a captured one."""
    import subprocess
    import sys
    code = f"""
import torch, synth, block_quantized_int8_mmq_gb300 as mmq
M, N, K = {M}, 512, 768
w = [torch.from_numpy(synth.weights("q4_k", i, N, K)).cuda() for i in (1, 2)]
x = torch.randn((M, K), device="cuda", dtype=torch.bfloat16)
gate, up = (torch.empty((M, N), device="cuda", dtype=torch.bfloat16) for _ in range(2))
torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    h = mmq.mmq_gated(x, w[0], w[1], "q4_k", N, gate=gate, up=up)
    dx = mmq.mmq_gated_backward(h, gate, up, w[0], w[1], "q4_k", K)
g.replay()
torch.cuda.synchronize()
a = mmq.mmq_gated(x, w[0], w[1], "q4_k", N)
b = mmq.mmq_gated_backward(a, gate, up, w[0], w[1], "q4_k", K)
assert torch.equal(a, h) and torch.equal(b, dx) and mmq.mmq_get_device_error() == 0
"""
    import os
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", code], cwd=root, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]


@pytest.mark.parametrize("M", [1, 5, 8, 9, 16])
@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("fmt", FMTS)
def test_few_rows_over_long_and_short_sums(fmt, dtype, M):
    """The stream of weights: x held in shared memory or not, one share of the reduction or sixteen, ragged columns."""
    for N, K in ((33, 256), (500, 4096), (2500, 1024), (40, 18944)):
        project(fmt, dtype, M, N, K, act="silu", bias=True, residual=True, seed=K + M)
    gated(fmt, dtype, M, 2450, 768, seed=M)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("N,K", [(20, 18944), (333, 13824), (1300, 13824), (3584, 9472)])
def test_few_columns_of_a_long_reduction(fmt, dtype, N, K):
    """Few rows: the reduction in one, two, four and eight CTAs; rows held in shared memory and rows that are not."""
    for M in (1, 11):
        project(fmt, dtype, M, N, K, seed=N + M)
    gated(fmt, dtype, 2, N // 4, K, seed=N)


@pytest.mark.parametrize("fmt", FMTS)
def test_clusters_in_a_graph_and_on_two_streams(fmt):
    """Reductions that CTAs share: replayed with other rows, and two calls at once, the bits of single calls; wide gradients too."""
    N, K, wide = 333, 13824, 5000
    w, back = Weights(fmt, 3, N, K), Weights(fmt, 4, wide, 256)
    xs = [rows(i, 3, K, "bf16") for i in range(2)]
    dys, zs = ([rows(i + k, 30, wide, "bf16") for i in range(2)] for k in (10, 20))
    run = lambda x, dy, z: (mmq.mmq_project(x, w.bytes, fmt, N), mmq.mmq_project_backward(dy, back.bytes, fmt, 256, act="silu", pre=z))
    want = [run(*t) for t in zip(xs, dys, zs)]
    kept = [t[0].clone() for t in (xs, dys, zs)]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = run(*kept)
    for i in (1, 0):
        for t, new in zip(kept, (xs[i], dys[i], zs[i])):
            t.copy_(new)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want[i]))
    sides = [torch.cuda.Stream() for _ in range(2)]
    outs = [[], []]
    for _ in range(4):
        for i, side in enumerate(sides):
            with torch.cuda.stream(side):
                outs[i].append(run(xs[i], dys[i], zs[i]))
    torch.cuda.synchronize()
    clean()
    assert all(torch.equal(a, b) for i in range(2) for o in outs[i] for a, b in zip(o, want[i]))


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("K", [512, 8704])
def test_few_f32_rows_keep_their_precision(fmt, K):
    """A block's products and its minimum's leave the tensor core after four cuts of 2^-24 of the largest product, which is a few
    times the block's sum: 16 x 2^-24 of the norm in all, beside the rows' own two terms (2^-23)."""
    N = 395
    w = Weights(fmt, 5, N, K)
    for M in (1, 14):
        x = rows(6, M, K, "f32")
        z = x.double() @ w.v.double().T
        y = mmq.mmq_project(x, w.bytes, fmt, N)
        clean()
        assert float((y.double() - z).norm() / z.norm()) <= 2.0 ** -20 + 2.0 ** -23


@pytest.mark.parametrize("dtype", ["f32", "f16"])
@pytest.mark.parametrize("N", [4090, 4100, 26000])
def test_wide_gradients(dtype, N):
    """Rows of gradients in small CTAs, in large ones, and too wide to be kept between their two looks."""
    backward("q8_0", dtype, 21, N, 64, 2, keep=True, seed=N)
    backward("q8_0", dtype, 3, N, 64, 1, act="gelu", keep=True, seed=N)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("M", [2, 30, 140])
def test_q6_k_rows_that_begin_on_16_bytes(dtype, M):
    """2048 and 4096 values: rows of a multiple of 16 bytes whose chunks of 210 are not."""
    for K in (2048, 4096):
        project("q6_k", dtype, M, 150, K, seed=K)
        backward("q6_k", dtype, M, 150, K, 2, seed=K)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_feed_forward_example(dtype):
    """The example runs and its gradients are right: a dozen roundings of the rows' type (half a step each, a few to a stage)
    and of the weights on the way, 24 half steps of bf16 in all; f32 as the tensor cores' products leave it, and torch's
    own f32 products of the adapter."""
    import importlib.util
    import os
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "feed_forward.py")
    spec = importlib.util.spec_from_file_location("feed_forward", path)
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    errors = example.run(tokens=90, steps=3, dtype=DT[dtype], quiet=True, hidden=512, inner=768)
    assert len(errors) == 5 and max(errors) <= (2.0 ** -16 if dtype == "f32" else 24 * 2.0 ** -8)


def test_profiler_names():
    w = Weights("q4_k", 1, 64, 256)
    prev = mmq.mmq_profile_enable(True)
    try:
        for M in (4, 40):
            mmq.mmq_project(rows(1, M, 256, "f16"), w.bytes, "q4_k", 64)
        mmq.mmq_project_backward(rows(1, 4, 64, "f16"), w.bytes, "q4_k", 256)
        torch.cuda.synchronize()
        names = mmq.mmq_profile_read(reset=True)
    finally:
        mmq.mmq_profile_enable(prev)
    assert {"k_ffn_rows", "k_ffn_stream", "k_ffn_tile", "k_ffn_gradients", "k_ffn_tile_back"} <= set(names)
