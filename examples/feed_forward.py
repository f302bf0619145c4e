"""The feed-forward half of a quantized layer, as a server runs it and as adapters are trained through it: the
gated block and the projection back into the residual stream, over block-quantized weights of two formats.

    python examples/feed_forward.py [--tokens 300] [--steps 16] [--dtype bfloat16]

A prompt goes through, then single tokens with the step captured in a CUDA graph.  Then a low-rank adapter on the
gate is trained for one step beside the frozen weights: its gradients come from the gradient of the gate that the way back
leaves, and the gradient of the block's input from that and the adapter's own.
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import block_quantized_int8_mmq_gb300 as mmq  # noqa: E402
import synth  # noqa: E402


class FeedForward:
    """x + (silu(x Wg^T) * (x Wu^T)) Wd^T: gate and up of one format, down of another."""

    def __init__(self, hidden=3584, inner=18944, fmt="q8_0", down="q6_k", seed=1):
        self.hidden, self.inner, self.fmt, self.down = hidden, inner, fmt, down
        self.w_gate, self.w_up = (torch.from_numpy(synth.weights(fmt, seed + i, inner, hidden)).cuda() for i in range(2))
        self.w_down = torch.from_numpy(synth.weights(down, seed + 2, hidden, inner)).cuda()

    def __call__(self, x, keep=None):
        gate, up = keep if keep is not None else (None, None)
        h = mmq.mmq_gated(x, self.w_gate, self.w_up, self.fmt, self.inner, gate=gate, up=up)
        return mmq.mmq_project(h, self.w_down, self.down, self.hidden, residual=x)

    def backward(self, dy, keep, dgate=None, dup=None):
        dh = mmq.mmq_project_backward(dy, self.w_down, self.down, self.inner)
        dx = mmq.mmq_gated_backward(dh, *keep, self.w_gate, self.w_up, self.fmt, self.hidden, dgate=dgate, dup=dup)
        return dx + dy  # the residual's way past the block


def weights_of(wq, fmt, N, K):
    """f64 [N, K] values of blocks, through the projection: the rows of the identity."""
    return mmq.mmq_project(torch.eye(K, device="cuda"), wq, fmt, N).double().T


def run(tokens=300, steps=16, dtype=torch.bfloat16, rank=8, quiet=False, **sizes):
    """Relative errors, against 64 bits, of the prompt's output, of the last step's, of the block's input gradient and
    of the adapter's two."""
    block = FeedForward(**sizes)
    K, N = block.hidden, block.inner
    gen = torch.Generator(device="cuda").manual_seed(7)
    x = torch.randn((tokens, K), device="cuda", generator=gen).to(dtype)
    wg, wu = (weights_of(w, block.fmt, N, K) for w in (block.w_gate, block.w_up))
    wd = weights_of(block.w_down, block.down, K, N)

    def plain(x):
        g = x @ wg.T
        return x + (g * torch.sigmoid(g) * (x @ wu.T)) @ wd.T

    def off(got, want):
        return float((got.double() - want).norm() / want.norm())
    errors = [off(block(x), plain(x.double()))]

    # single tokens: what one step gives, brought back to size, is the next one's input
    row, y = x[-1:].clone(), torch.empty((1, K), dtype=dtype, device="cuda")
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        before = row.clone()
        y.copy_(block(row))
        row.copy_(y / y.float().square().mean().sqrt())
    for _ in range(steps):
        graph.replay()
    torch.cuda.synchronize()
    errors.append(off(y, plain(before.double())))

    # one step of an adapter on the gate, g += (x A^T) B^T.  B starts at zero, so the forward pass is the block's own and
    # A's gradient is zero; here both are small and their part of the gate is added to what the block keeps
    A = (torch.randn((rank, K), device="cuda", generator=gen) * 0.02).to(dtype)
    B = (torch.randn((N, rank), device="cuda", generator=gen) * 0.02).to(dtype)
    keep = [torch.empty((tokens, N), dtype=dtype, device="cuda") for _ in range(2)]
    mmq.mmq_gated(x, block.w_gate, block.w_up, block.fmt, N, gate=keep[0], up=keep[1])
    xa = x @ A.T
    keep[0] += xa @ B.T
    dy = torch.randn((tokens, K), device="cuda", generator=gen).to(dtype)
    dgate = torch.empty((tokens, N), dtype=dtype, device="cuda")
    dx = block.backward(dy, keep, dgate=dgate)
    dB = dgate.T @ xa
    dxa = dgate @ B
    dA, dx = dxa.T @ x, dx + dxa @ A
    assert mmq.mmq_get_device_error() == 0

    # the same by 64-bit automatic differentiation from what was kept
    xd, Ad, Bd = (t.double().requires_grad_() for t in (x, A, B))
    g = xd @ wg.T + (xd @ Ad.T) @ Bd.T
    out = xd + (g * torch.sigmoid(g) * (xd @ wu.T)) @ wd.T
    for got, want in zip((dx, dA, dB), torch.autograd.grad(out, (xd, Ad, Bd), dy.double())):
        errors.append(off(got, want))
    if not quiet:
        names = ("prompt", "last token", "dx", "dA", "dB")
        print(f"{K} -> {N} -> {K}, {tokens} tokens, {dtype}: " + ", ".join(f"{n} {e:.1e}" for n, e in zip(names, errors)) + " off")
    return errors


if __name__ == "__main__":
    p = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    p.add_argument("--tokens", type=int, default=300)
    p.add_argument("--steps", type=int, default=16)
    p.add_argument("--dtype", default="bfloat16", choices=["float32", "bfloat16", "float16"])
    a = p.parse_args()
    run(a.tokens, a.steps, getattr(torch, a.dtype))
