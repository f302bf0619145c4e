"""Feed-forward operators over block-quantized weights (include/mmq.h, "feed-forward operators"): the
projection with bias, activation and residual in its epilogue, the gated block, and the way back of
both to their inputs.

    h = mmq_gated(x, w_gate, w_up, "q4_k", N)                       # silu(x Wg^T) * (x Wu^T)
    y = mmq_project(h, w_down, "q6_k", K, residual=r)               # h Wd^T + r
    dh = mmq_project_backward(dy, w_down, "q6_k", N)                # dy Wd
    dx = mmq_gated_backward(dh, gate, up, w_gate, w_up, "q4_k", K)  # gate, up: kept by mmq_gated

Rows are float32, bfloat16 or float16 and enter unquantized; weights are uint8 blocks as for mmq_gemm_*.
The tensors' device has to be the current one.  The calls do not record themselves for autograd: outputs carry no
graph, whether inputs require gradients or not, and a program that wants one calls the ways back from a
torch.autograd.Function of its own (examples/feed_forward.py has one).
"""
from __future__ import annotations

import ctypes

import torch

from . import MMQError, _lib
from .kv import _DTYPES, _empty, _stream_of

ACTS = {None: 0, "none": 0, "silu": 1, "gelu": 2, "gelu_tanh": 3, "relu": 4}


def _bind():
    P, I64, I = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int
    _lib.mmq_project.argtypes = [I, I, P, I64, I64, P, I64, I64, P, I, P, I64, P, P, P]
    _lib.mmq_gated.argtypes = [I, I, P, I64, I64, P, P, I64, I64, P, P, I, P, P, P, P]
    _lib.mmq_project_backward.argtypes = [I, I, P, I64, I64, P, I64, I64, I, P, P, P, P]
    _lib.mmq_gated_backward.argtypes = [I, I, P, I64, I64, P, P, I64, I64, I, P, P, P, P, P, P]


_bind()


_BLOCK = {"q8_0": (0, 34, 32), "q4_k": (1, 144, 256), "q5_k": (2, 176, 256), "q6_k": (3, 210, 256)}


def _refuse_rows(t, what):
    """Why a call's leading array is refused."""
    if not t.is_cuda or t.dtype not in _DTYPES:
        raise ValueError(f"{what} is {t.dtype} on {t.device}: float32, bfloat16 and float16 on a GPU are taken")
    if t.dim() != 2:
        raise ValueError(f"{what} has shape {tuple(t.shape)}: [rows, width] is wanted")
    raise ValueError(f"{what}: the last axis must be contiguous")


def _rows(t, what):
    """(dtype code, device, rows, width, stride) of the leading array of a call: [rows, width] on the current device,
    its rows contiguous.  A single row has no stride."""
    shape, dt, dev = t.shape, _DTYPES.get(t.dtype), t.device
    if dt is None or len(shape) != 2 or dev.type != "cuda":
        _refuse_rows(t, what)
    stride, step = t.stride()
    if step != 1 and shape[1] > 1:
        _refuse_rows(t, what)
    current = torch.cuda.current_device()
    if current != dev.index:
        raise ValueError(f"{what} is on {dev}, the current device is cuda:{current}: call it under "
                         f"torch.cuda.device({dev.index})")
    return dt, dev, shape[0], shape[1], stride if shape[0] > 1 else shape[1]


def _like(t, x, shape, what):
    """An array of the call's type that is read with a row stride: its address and stride."""
    if t is None:
        return None, 0
    if t.dtype != x.dtype or t.device != x.device or t.shape != shape or (shape[1] > 1 and t.stride(1) != 1):
        raise ValueError(f"{what} must be a {x.dtype} {tuple(shape)} tensor on {x.device} with a contiguous last axis")
    return t.data_ptr(), t.stride(0) if shape[0] > 1 else shape[1]


def _whole(t, x, shape, what):
    """A contiguous array of the call's type, or None."""
    if t is None:
        return None
    if t.dtype != x.dtype or t.device != x.device or t.shape != shape or not t.is_contiguous():
        raise ValueError(f"{what} must be a contiguous {x.dtype} {tuple(shape)} tensor on {x.device}")
    return t.data_ptr()


def _bias(t, x, N, what):
    if t is None:
        return None
    if t.dtype != torch.float32 or t.device != x.device or t.shape != (N,) or not t.is_contiguous():
        raise ValueError(f"{what} must be a contiguous float32 [{N}] tensor on {x.device}")
    return t.data_ptr()


def _format(fmt, N, K):
    """The format's code and the bytes of an [N, K] matrix (0 where K is no whole number of blocks)."""
    b = _BLOCK.get(fmt)
    if b is None:
        raise ValueError(f"fmt {fmt!r}: one of {', '.join(_BLOCK)} is taken")
    return b[0], 0 if K % b[2] else N * (K // b[2]) * b[1]


def _weight(t, x, nbytes, what):
    if t.dtype != torch.uint8 or t.device != x.device or not t.is_contiguous() or t.numel() != nbytes:
        raise ValueError(f"{what} must be a contiguous uint8 tensor of {nbytes} bytes on {x.device}, got "
                         f"{t.numel()} {t.dtype} on {t.device}")
    return t.data_ptr()


def _act(act):
    a = ACTS.get(act)
    if a is None:
        raise ValueError(f"act {act!r}: one of {', '.join(k for k in ACTS if k)} is taken")
    return a


def _result(t, x, shape, dev, stream, what):
    """Where a call's result goes: the tensor given, or one of its own."""
    if t is None:
        t = _empty(shape, x.dtype, dev, stream)
    elif t.dtype != x.dtype or t.device != dev or t.shape != shape or not t.is_contiguous():
        raise ValueError(f"{what} must be a contiguous {x.dtype} {tuple(shape)} tensor on {dev}")
    return t


def mmq_project(x, wq, fmt: str, N: int, bias=None, act=None, residual=None, pre=None, out=None, stream=None):
    """act(x W^T + bias) + residual: x [M, K] rows, wq [N, ...] blocks, bias f32 [N], residual [M, N] (it may
    be `out`).  act: "silu", "gelu", "gelu_tanh", "relu" or None.  pre: a tensor [M, N] for x W^T + bias."""
    dt, dev, M, K, stride = _rows(x, "x")
    shape = (M, N)
    f, nbytes = _format(fmt, N, K)
    a, w, b = _act(act), _weight(wq, x, nbytes, "wq"), _bias(bias, x, N, "bias")
    r, rs = _like(residual, x, shape, "residual")
    p = _whole(pre, x, shape, "pre")
    out = _result(out, x, shape, dev, stream, "out")
    st = _lib.mmq_project(f, dt, x.data_ptr(), stride, M, w, N, K, b, a, r, rs, p, out.data_ptr(), _stream_of(dev, stream))
    if st != 0:
        raise MMQError("mmq_project", st)
    return out


def mmq_gated(x, w_gate, w_up, fmt: str, N: int, act="silu", bias_gate=None, bias_up=None, gate=None, up=None, out=None,
              stream=None):
    """act(x Wg^T + bg) * (x Wu^T + bu): x [M, K] rows, w_gate and w_up [N, ...] blocks.  gate, up: tensors
    [M, N] for the two projections, which the backward pass takes."""
    dt, dev, M, K, stride = _rows(x, "x")
    shape = (M, N)
    f, nbytes = _format(fmt, N, K)
    a, wg, wu = _act(act), _weight(w_gate, x, nbytes, "w_gate"), _weight(w_up, x, nbytes, "w_up")
    bg, bu = _bias(bias_gate, x, N, "bias_gate"), _bias(bias_up, x, N, "bias_up")
    g, u = _whole(gate, x, shape, "gate"), _whole(up, x, shape, "up")
    out = _result(out, x, shape, dev, stream, "out")
    st = _lib.mmq_gated(f, dt, x.data_ptr(), stride, M, wg, wu, N, K, bg, bu, a, g, u, out.data_ptr(), _stream_of(dev, stream))
    if st != 0:
        raise MMQError("mmq_gated", st)
    return out


def mmq_project_backward(dy, wq, fmt: str, K: int, act=None, pre=None, dz=None, dx=None, stream=None):
    """The gradient of mmq_project's x: (dy act'(pre)) W, [M, K], from dy [M, N].  pre: what mmq_project kept
    (needed where there is an activation).  dz: a tensor [M, N] for dy act'(pre)."""
    dt, dev, M, N, stride = _rows(dy, "dy")
    f, nbytes = _format(fmt, N, K)
    a, w = _act(act), _weight(wq, dy, nbytes, "wq")
    p, z = _whole(pre, dy, (M, N), "pre"), _whole(dz, dy, (M, N), "dz")
    dx = _result(dx, dy, (M, K), dev, stream, "dx")
    st = _lib.mmq_project_backward(f, dt, dy.data_ptr(), stride, M, w, N, K, a, p, z, dx.data_ptr(), _stream_of(dev, stream))
    if st != 0:
        raise MMQError("mmq_project_backward", st)
    return dx


def mmq_gated_backward(dh, gate, up, w_gate, w_up, fmt: str, K: int, act="silu", dgate=None, dup=None, dx=None,
                       stream=None):
    """The gradient of mmq_gated's x, [M, K], from dh [M, N] and the gate and up that mmq_gated kept.  dgate, dup:
    tensors [M, N] for the gradients of gate and up."""
    dt, dev, M, N, stride = _rows(dh, "dh")
    f, nbytes = _format(fmt, N, K)
    shape = (M, N)
    a, wg, wu = _act(act), _weight(w_gate, dh, nbytes, "w_gate"), _weight(w_up, dh, nbytes, "w_up")
    g, u = _whole(gate, dh, shape, "gate"), _whole(up, dh, shape, "up")
    dg, du = _whole(dgate, dh, shape, "dgate"), _whole(dup, dh, shape, "dup")
    dx = _result(dx, dh, (M, K), dev, stream, "dx")
    st = _lib.mmq_gated_backward(f, dt, dh.data_ptr(), stride, M, wg, wu, N, K, a, g, u, dg, du, dx.data_ptr(),
                                 _stream_of(dev, stream))
    if st != 0:
        raise MMQError("mmq_gated_backward", st)
    return dx
