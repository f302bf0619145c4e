"""The feed-forward operators from their definition, in 64 bits (torch, any device): what blocks stand for,
value by value, the activations with their derivatives, the products, and the sums that error bounds need."""
import math

import numpy as np
import torch

BYTES = {"q8_0": 34, "q4_k": 144, "q5_k": 176, "q6_k": 210}
ACTS = ("none", "silu", "gelu", "gelu_tanh", "relu")


def _f16(lo, hi):
    return (lo.astype(np.uint16) | hi.astype(np.uint16) << 8).view(np.float16).astype(np.float64)


def values(fmt, w):
    """(values, sizes) f64 [N, K] of blocks uint8 [N, row bytes]: what each weight stands for, and the sum of
    the magnitudes that it is formed from (code x scale, and the block's minimum)."""
    w = np.ascontiguousarray(w)
    b = w.reshape(w.shape[0], -1, BYTES[fmt])
    if fmt == "q8_0":
        v = b[..., 2:].view(np.int8) * _f16(b[..., 0], b[..., 1])[..., None]
        v = v.reshape(w.shape[0], -1)
        return v, np.abs(v)
    out, size = np.empty((*b.shape[:2], 256)), np.empty((*b.shape[:2], 256))
    for v in range(256):
        if fmt == "q6_k":
            h, t, l = v // 128, v % 128 // 32, v % 32
            q = (b[..., 64 * h + 32 * (t % 2) + l] >> 4 * (t // 2)) & 15
            q = q + 16.0 * ((b[..., 128 + 32 * h + l] >> 2 * t) & 3) - 32
            out[..., v] = q * b[..., 192 + v // 16].view(np.int8) * _f16(b[..., 208], b[..., 209])
            size[..., v] = np.abs(out[..., v])
            continue
        c, h, i, j = v // 64, v % 64 // 32, v % 32, v // 32
        q = (b[..., (16 if fmt == "q4_k" else 48) + 32 * c + i] >> 4 * h) & 15
        if fmt == "q5_k":
            q = q + 16 * ((b[..., 16 + i] >> 2 * c + h) & 1)
        if j < 4:
            sc, mn = b[..., 4 + j] & 63, b[..., 8 + j] & 63
        else:
            sc, mn = (b[..., 8 + j] & 15) | b[..., j] >> 6 << 4, b[..., 8 + j] >> 4 | b[..., 4 + j] >> 6 << 4
        part, least = q * (sc * _f16(b[..., 0], b[..., 1])), mn * _f16(b[..., 2], b[..., 3])
        out[..., v], size[..., v] = part - least, np.abs(part) + np.abs(least)
    return out.reshape(w.shape[0], -1), size.reshape(w.shape[0], -1)


def act(name, z):
    """act(z) and act'(z) of f64 z."""
    if name == "none":
        return z, torch.ones_like(z)
    if name == "relu":
        return z.clamp(min=0), (z > 0).double()
    if name == "silu":
        s = torch.sigmoid(z)
        return z * s, s * (1 + z * (1 - s))
    if name == "gelu":
        s = (1 + torch.erf(z / math.sqrt(2))) / 2
        return z * s, s + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)
    c = math.sqrt(2 / math.pi)
    t = torch.tanh(c * (z + 0.044715 * z ** 3))
    return z * (1 + t) / 2, (1 + t) / 2 + z / 2 * (1 - t * t) * c * (1 + 3 * 0.044715 * z * z)
