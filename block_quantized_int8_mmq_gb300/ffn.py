"""Feed-forward operators over block-quantized weights (include/mmq.h, "feed-forward operators"): the
projection with bias, activation and residual in its epilogue, the gated block, and the way back of
both to their inputs.

    h = mmq_gated(x, w_gate, w_up, "q4_k", N)                       # silu(x Wg^T) * (x Wu^T)
    y = mmq_project(h, w_down, "q6_k", K, residual=r)               # h Wd^T + r
    dh = mmq_project_backward(dy, w_down, "q6_k", N)                # dy Wd
    dx = mmq_gated_backward(dh, gate, up, w_gate, w_up, "q4_k", K)  # gate, up: kept by mmq_gated

Rows are float32, bfloat16 or float16 and enter unquantized; weights are uint8 blocks as for mmq_gemm_*.
The tensors' device has to be the current one.
"""
from __future__ import annotations

import ctypes

import torch

from . import FMT, MMQError, _lib, mmq_weight_row_bytes
from .kv import _DTYPES, _empty, _stream_of

ACTS = {"none": 0, "silu": 1, "gelu": 2, "gelu_tanh": 3, "relu": 4}


def _bind():
    P, I64, I = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int
    _lib.mmq_project.argtypes = [I, I, P, I64, I64, P, I64, I64, P, I, P, I64, P, P, P]
    _lib.mmq_gated.argtypes = [I, I, P, I64, I64, P, P, I64, I64, P, P, I, P, P, P, P]
    _lib.mmq_project_backward.argtypes = [I, I, P, I64, I64, P, I64, I64, I, P, P, P, P]
    _lib.mmq_gated_backward.argtypes = [I, I, P, I64, I64, P, P, I64, I64, I, P, P, P, P, P, P]


_bind()


def _rows(t, what, width=None):
    """The leading array of a call: [rows, width] on the current device, its rows contiguous."""
    if not t.is_cuda or t.dtype not in _DTYPES:
        raise ValueError(f"{what} is {t.dtype} on {t.device}: float32, bfloat16 and float16 on a GPU are taken")
    if t.dim() != 2 or (width is not None and t.shape[1] != width):
        raise ValueError(f"{what} has shape {tuple(t.shape)}: [rows, {'width' if width is None else width}] is wanted")
    if t.shape[1] > 1 and t.stride(1) != 1:
        raise ValueError(f"{what}: the last axis must be contiguous")
    current = torch.cuda.current_device()
    if current != t.device.index:
        raise ValueError(f"{what} is on {t.device}, the current device is cuda:{current}: call it under "
                         f"torch.cuda.device({t.device.index})")
    return _DTYPES[t.dtype]


def _stride(t):
    """Elements from row to row (a single row has none)."""
    return t.stride(0) if t.shape[0] > 1 else t.shape[1]


def _like(t, x, shape, what):
    """An array of the call's type that is read with a row stride, or None."""
    if t is None:
        return None
    if t.dtype != x.dtype or t.device != x.device or t.shape != shape or (shape[1] > 1 and t.stride(1) != 1):
        raise ValueError(f"{what} must be a {x.dtype} {tuple(shape)} tensor on {x.device} with a contiguous last axis")
    return t.data_ptr()


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


def _weight(t, x, nbytes, what):
    if t.dtype != torch.uint8 or t.device != x.device or not t.is_contiguous() or t.numel() != nbytes:
        raise ValueError(f"{what} must be a contiguous uint8 tensor of {nbytes} bytes on {x.device}, got "
                         f"{t.numel()} {t.dtype} on {t.device}")
    return t.data_ptr()


def _act(act):
    a = ACTS.get("none" if act is None else act)
    if a is None:
        raise ValueError(f"act {act!r}: one of {', '.join(ACTS)} is taken")
    return a


def _fmt(fmt):
    f = FMT.get(fmt)
    if f is None:
        raise ValueError(f"fmt {fmt!r}: one of {', '.join(FMT)} is taken")
    return f


def _check(fn, st):
    if st != 0:
        raise MMQError(fn, st)


def mmq_project(x, wq, fmt: str, N: int, bias=None, act=None, residual=None, pre=None, out=None, stream=None):
    """act(x W^T + bias) + residual: x [M, K] rows, wq [N, ...] blocks, bias f32 [N], residual [M, N] (it may
    be `out`).  act: "silu", "gelu", "gelu_tanh", "relu" or None.  pre: a tensor [M, N] for x W^T + bias."""
    dt = _rows(x, "x")
    M, K = x.shape
    shape, f = (M, N), _fmt(fmt)
    w = _weight(wq, x, N * mmq_weight_row_bytes(fmt, K), "wq")
    b, p = _bias(bias, x, N, "bias"), _whole(pre, x, shape, "pre")
    r = _like(residual, x, shape, "residual")
    if out is None:
        out = _empty(shape, x.dtype, x.device, stream)
    o = _whole(out, x, shape, "out")
    _check("mmq_project", _lib.mmq_project(f, dt, x.data_ptr(), _stride(x), M, w, N, K, b, _act(act), r,
                                           0 if r is None else _stride(residual), p, o, _stream_of(x.device, stream)))
    return out


def mmq_gated(x, w_gate, w_up, fmt: str, N: int, act="silu", bias_gate=None, bias_up=None, gate=None, up=None, out=None,
              stream=None):
    """act(x Wg^T + bg) * (x Wu^T + bu): x [M, K] rows, w_gate and w_up [N, ...] blocks.  gate, up: tensors
    [M, N] for the two projections, which the backward pass takes."""
    dt = _rows(x, "x")
    M, K = x.shape
    shape, f, nbytes = (M, N), _fmt(fmt), N * mmq_weight_row_bytes(fmt, K)
    wg, wu = _weight(w_gate, x, nbytes, "w_gate"), _weight(w_up, x, nbytes, "w_up")
    bg, bu = _bias(bias_gate, x, N, "bias_gate"), _bias(bias_up, x, N, "bias_up")
    g, u = _whole(gate, x, shape, "gate"), _whole(up, x, shape, "up")
    if out is None:
        out = _empty(shape, x.dtype, x.device, stream)
    o = _whole(out, x, shape, "out")
    _check("mmq_gated", _lib.mmq_gated(f, dt, x.data_ptr(), _stride(x), M, wg, wu, N, K, bg, bu, _act(act), g, u, o,
                                       _stream_of(x.device, stream)))
    return out


def mmq_project_backward(dy, wq, fmt: str, K: int, act=None, pre=None, dz=None, dx=None, stream=None):
    """The gradient of mmq_project's x: (dy act'(pre)) W, [M, K], from dy [M, N].  pre: what mmq_project kept
    (needed where there is an activation).  dz: a tensor [M, N] for dy act'(pre)."""
    dt = _rows(dy, "dy")
    M, N = dy.shape
    f, a = _fmt(fmt), _act(act)
    w = _weight(wq, dy, N * mmq_weight_row_bytes(fmt, K), "wq")
    p, z = _whole(pre, dy, (M, N), "pre"), _whole(dz, dy, (M, N), "dz")
    if dx is None:
        dx = _empty((M, K), dy.dtype, dy.device, stream)
    o = _whole(dx, dy, (M, K), "dx")
    _check("mmq_project_backward", _lib.mmq_project_backward(f, dt, dy.data_ptr(), _stride(dy), M, w, N, K, a, p, z, o,
                                                             _stream_of(dy.device, stream)))
    return dx


def mmq_gated_backward(dh, gate, up, w_gate, w_up, fmt: str, K: int, act="silu", dgate=None, dup=None, dx=None,
                       stream=None):
    """The gradient of mmq_gated's x, [M, K], from dh [M, N] and the gate and up that mmq_gated kept.  dgate, dup:
    tensors [M, N] for the gradients of gate and up."""
    dt = _rows(dh, "dh")
    M, N = dh.shape
    f, a, shape, nbytes = _fmt(fmt), _act(act), (M, N), N * mmq_weight_row_bytes(fmt, K)
    wg, wu = _weight(w_gate, dh, nbytes, "w_gate"), _weight(w_up, dh, nbytes, "w_up")
    g, u = _whole(gate, dh, shape, "gate"), _whole(up, dh, shape, "up")
    dg, du = _whole(dgate, dh, shape, "dgate"), _whole(dup, dh, shape, "dup")
    if dx is None:
        dx = _empty((M, K), dh.dtype, dh.device, stream)
    o = _whole(dx, dh, (M, K), "dx")
    _check("mmq_gated_backward", _lib.mmq_gated_backward(f, dt, dh.data_ptr(), _stride(dh), M, wg, wu, N, K, a, g, u, dg,
                                                         du, o, _stream_of(dh.device, stream)))
    return dx
