"""The feed-forward operators without a GPU: the refusals of their C entry points (nothing is launched, so any
aligned address stands for device memory), those of the binding, and the reference the GPU tests compare with."""
import ctypes

import numpy as np
import pytest

import oracle
import synth

mmq = pytest.importorskip("block_quantized_int8_mmq_gb300")
torch = pytest.importorskip("torch")
import ffn_ref  # noqa: E402
from block_quantized_int8_mmq_gb300 import ffn  # noqa: E402, F401  (binds the entry points)

SHAPE, KMUL, NULL, ALIGN, ARG = -1, -2, -3, -4, -9
A = 1 << 20
FNS = ["project", "gated", "project_backward", "gated_backward"]


def call(fn, **change):
    """One of the entries on well-formed arguments (no rows) but for `change`."""
    f = dict(fmt=1, dtype=0, x=A, xs=None, M=0, w=A, w2=A, N=24, K=256, bias=A, bias2=A, act=1, residual=A, rs=None, pre=A,
             up=A, dz=A, dup=A, out=A)
    f.update(change)
    back = fn.endswith("backward")
    xs = f["xs"] if f["xs"] is not None else f["N"] if back else f["K"]
    rs = f["rs"] if f["rs"] is not None else f["N"]
    head = (f["fmt"], f["dtype"], f["x"], xs, f["M"], f["w"])
    L = mmq.lib()
    if fn == "project":
        return L.mmq_project(*head, f["N"], f["K"], f["bias"], f["act"], f["residual"], rs, f["pre"], f["out"], None)
    if fn == "gated":
        return L.mmq_gated(*head, f["w2"], f["N"], f["K"], f["bias"], f["bias2"], f["act"], f["pre"], f["up"], f["out"], None)
    if fn == "project_backward":
        return L.mmq_project_backward(*head, f["N"], f["K"], f["act"], f["pre"], f["dz"], f["out"], None)
    return L.mmq_gated_backward(*head, f["w2"], f["N"], f["K"], f["act"], f["pre"], f["up"], f["dz"], f["dup"], f["out"], None)


@pytest.mark.parametrize("fn", FNS)
def test_no_rows_is_no_work(fn):
    for fmt in range(4):
        assert call(fn, fmt=fmt) == 0
    assert call(fn, fmt=0, K=32) == call(fn, x=None, out=None) == call(fn, act=0) == 0
    if fn.endswith("backward"):
        assert call(fn, dz=None, dup=None) == 0
    else:
        assert call(fn, bias=None, bias2=None, pre=None, up=None, residual=None) == 0


@pytest.mark.parametrize("fn", FNS)
@pytest.mark.parametrize("change,status", [
    (dict(fmt=4), ARG), (dict(fmt=-1), ARG), (dict(dtype=3), ARG), (dict(dtype=-1), ARG), (dict(act=5), ARG), (dict(act=-1), ARG),
    (dict(M=-1), SHAPE), (dict(N=0), SHAPE), (dict(K=0), SHAPE), (dict(K=128), KMUL), (dict(fmt=0, K=48), KMUL),
    (dict(M=1 << 31), SHAPE), (dict(N=1 << 31), SHAPE), (dict(M=1 << 29, N=1 << 12), SHAPE), (dict(N=1 << 29, K=1 << 12), SHAPE),
    (dict(M=1 << 29, K=1 << 12), SHAPE), (dict(w=None), NULL), (dict(w=A + 8), ALIGN), (dict(x=None, M=1), NULL),
    (dict(out=None, M=1), NULL), (dict(out=A + 2), ALIGN), (dict(dtype=1, out=A + 1), ALIGN), (dict(x=A + 2), ALIGN),
    (dict(xs=23, M=2), SHAPE), (dict(xs=1 << 41), SHAPE), (dict(pre=A + 1), ALIGN)])
def test_refusals(fn, change, status, capfd):
    assert call(fn, **change) == status
    assert f"mmq_{fn} refused" in capfd.readouterr().err


@pytest.mark.parametrize("fn,change,status", [
    ("project", dict(x=A + 8), ALIGN), ("gated", dict(x=A + 4), ALIGN), ("project", dict(xs=258, M=2), ALIGN),
    ("gated", dict(dtype=2, xs=260, M=2), ALIGN), ("project", dict(bias=A + 2), ALIGN), ("gated", dict(bias=A + 1), ALIGN),
    ("gated", dict(bias2=A + 2), ALIGN), ("gated", dict(w2=None), NULL), ("gated", dict(w2=A + 4), ALIGN),
    ("gated", dict(up=A + 2), ALIGN), ("project", dict(residual=A + 2), ALIGN), ("project", dict(rs=23), SHAPE),
    ("gated_backward", dict(w2=None), NULL), ("gated_backward", dict(pre=None, M=1), NULL),
    ("gated_backward", dict(up=None, M=1), NULL), ("gated_backward", dict(up=A + 2), ALIGN),
    ("gated_backward", dict(dup=A + 2), ALIGN), ("project_backward", dict(pre=None, M=1), NULL),
    ("project_backward", dict(dz=A + 2), ALIGN), ("gated_backward", dict(act=0, pre=None, M=1), NULL)])
def test_refusals_of_each_call(fn, change, status, capfd):
    assert call(fn, **change) == status
    assert f"mmq_{fn} refused" in capfd.readouterr().err


def test_binding_refuses_what_is_not_on_a_gpu():
    x, w = torch.zeros((2, 256)), torch.zeros((4, 144), dtype=torch.uint8)
    with pytest.raises(ValueError, match="on a GPU"):
        mmq.mmq_project(x, w, "q4_k", 4)
    with pytest.raises(ValueError, match="on a GPU"):
        mmq.mmq_gated(x, w, w, "q4_k", 4)
    with pytest.raises(ValueError, match="on a GPU"):
        mmq.mmq_project_backward(x, w, "q4_k", 256)
    with pytest.raises(ValueError, match="on a GPU"):
        mmq.mmq_gated_backward(x, x, x, w, w, "q4_k", 256)


@pytest.mark.parametrize("fmt", ["q8_0", "q4_k", "q5_k", "q6_k"])
def test_reference_values_are_the_oracle_s(fmt):
    """One-hot rows of 127 have d = 1 and the code 127: the contraction gives 127 times each weight."""
    N, K = 3, 512
    w = synth.weights(fmt, 11, N, K)
    x = np.zeros((K, K), np.float32)
    np.fill_diagonal(x, 127.0)
    want, _ = oracle.gemm(fmt, oracle.quantize_q8_1(x), w, K, N, K)
    got, size = ffn_ref.values(fmt, w)
    assert np.abs(want.T / 127 - got).max() <= 2.0 ** -40 * np.abs(got).max()  # f64 sums of a few terms
    assert (size >= np.abs(got) * (1 - 2.0 ** -50)).all()


def test_reference_activations():
    z = torch.tensor([-3.0, -1.0, -0.25, 0.5, 2.0], dtype=torch.float64, requires_grad=True)
    by_hand = {"silu": 2 / (1 + np.exp(-2.0)), "gelu": 2 * 0.977249868051821, "gelu_tanh": 1.954597694087775, "relu": 2.0,
               "none": 2.0}
    for name in ffn_ref.ACTS:
        a, d = ffn_ref.act(name, z)
        assert abs(float(a[-1].detach()) - by_hand[name]) < 1e-14
        grad, = torch.autograd.grad(a.sum(), z)
        assert float((grad - d).abs().max()) < 1e-14
    assert float(ffn_ref.act("relu", torch.zeros(1, dtype=torch.float64))[1]) == 0
