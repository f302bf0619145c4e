"""The attention half of a quantized 7B GQA layer, as a server runs it: one joint projection of
queries, keys and values (block-quantized weights), the rotated keys and values appended to the
8-bit cache, attention over the cache, and the output projection.

    python examples/attention_layer.py [--fmt q4_k] [--prompts 300 77] [--steps 16]

The prompts (of different lengths) go through in one batch, then every sequence takes `steps`
single tokens with the whole step captured in a CUDA graph: the captured calls read lengths and
page tables from device memory, so one graph serves every step.  At the end the last step's
attention is checked against a plain one over the values that the cache holds.
"""
import argparse
import os
import sys
import time

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import block_quantized_int8_mmq_gb300 as mmq  # noqa: E402
import synth  # noqa: E402


class AttentionLayer:
    def __init__(self, fmt, hidden=3584, heads=28, kv_heads=4, dim=128, seed=1):
        self.fmt, self.hidden, self.heads, self.kv_heads, self.dim = fmt, hidden, heads, kv_heads, dim
        self.qkv_rows = (heads + 2 * kv_heads) * dim
        self.w_qkv = torch.from_numpy(synth.weights(fmt, seed, self.qkv_rows, hidden)).cuda()
        self.w_out = torch.from_numpy(synth.weights(fmt, seed + 1, hidden, heads * dim)).cuda()

    def __call__(self, x, cache, batch, rope, workspace=None):
        """x: f32 [tokens, hidden] -> f32 [tokens, hidden], and the attention's own output and queries."""
        T, H, KH, D = x.shape[0], self.heads, self.kv_heads, self.dim
        qkv = mmq.mmq_linear(x, self.w_qkv, self.fmt, self.qkv_rows)
        q, k, v = (qkv[:, a * D:b * D].view(T, -1, D) for a, b in ((0, H), (H, H + KH), (H + KH, H + 2 * KH)))
        q = mmq.mmq_kv_append(cache, batch, k, v, q=q, rope=rope)
        o = mmq.mmq_kv_attend(cache, batch, q, workspace=workspace)
        return mmq.mmq_linear(o.view(T, H * D), self.w_out, self.fmt, self.hidden), o, q


def int32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def plain_attention(q, k, v):
    """One row's attention in f64: q [heads, dim], k and v [tokens, kv heads, dim]."""
    g = q.shape[0] // k.shape[1]
    s = torch.einsum("hd,thd->ht", q.double(), k.double().repeat_interleave(g, 1)) / q.shape[-1] ** 0.5
    return torch.einsum("ht,thd->hd", s.softmax(-1), v.double().repeat_interleave(g, 1))


def run(fmt="q4_k", prompts=(300, 77), steps=16, page=64, quiet=False, **sizes):
    layer = AttentionLayer(fmt, **sizes)
    B, longest = len(prompts), max(prompts) + steps
    pages = -(-longest // page)
    cache = mmq.KVCache.empty(B * pages + 1, layer.kv_heads, layer.dim, page=page)
    table = torch.randperm(B * pages, device="cuda").view(B, pages).to(torch.int32)  # pages lie anywhere
    freq = 10000.0 ** (-torch.arange(0, layer.dim, 2, device="cuda", dtype=torch.float64) / layer.dim)
    angle = torch.arange(pages * page, device="cuda")[:, None] * freq
    rope = mmq.Rope(angle.cos().float(), angle.sin().float())
    gen = torch.Generator(device="cuda").manual_seed(5)

    # the prompts, packed one after another
    lens = int32(list(prompts))
    starts = [0]
    for n in prompts:
        starts.append(starts[-1] + n)
    x = torch.randn((starts[-1], layer.hidden), device="cuda", generator=gen)
    # random weights have no scale of their own: inputs for which queries and keys are of order one
    small = 1.0 / float(mmq.mmq_linear(x, layer.w_qkv, fmt, layer.qkv_rows).square().mean().sqrt())
    x.mul_(small)
    prefill = mmq.KVBatch(int32(starts), lens, table, starts[-1], max(prompts))
    layer(x, cache, prefill, rope)

    # single tokens: the graph's tensors stay, their contents change
    x = torch.randn((B, layer.hidden), device="cuda", generator=gen) * small
    step = mmq.KVBatch(int32(list(range(B + 1))), lens, table, B, 1)
    workspace = torch.zeros(mmq.mmq_kv_workspace_bytes(layer.dim), dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        lens.add_(1)
        y, o, q = layer(x, cache, step, rope, workspace)
        x.copy_(y * (small / y.square().mean(-1, keepdim=True).sqrt()))  # what the next step reads
    torch.cuda.synchronize()
    t0 = time.perf_counter()
    for _ in range(steps):
        graph.replay()
    torch.cuda.synchronize()
    took = time.perf_counter() - t0
    assert mmq.mmq_get_device_error() == 0

    # the last step against a plain attention over what the cache holds
    off = []
    for b, n in enumerate(prompts):
        whole = mmq.KVBatch(int32([0, n + steps]), int32([n + steps]), table[b:b + 1], n + steps, n + steps)
        k, v = mmq.mmq_kv_read(cache, whole)
        want = plain_attention(q[b], k, v)
        off.append(float((o[b].double() - want).norm() / want.norm()))
    worst = max(off, key=lambda e: (e != e, e))  # a NaN above all
    if not quiet:
        print(f"{fmt}: prompts of {list(prompts)} tokens, {steps} steps of {B} in {took * 1e3:.2f} ms "
              f"({took / steps * 1e6:.1f} us a step), last step {worst:.1e} off a plain attention")
    return worst


if __name__ == "__main__":
    p = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    p.add_argument("--fmt", default="q4_k", choices=["q8_0", "q4_k", "q5_k", "q6_k"])
    p.add_argument("--prompts", type=int, nargs="+", default=[300, 77])
    p.add_argument("--steps", type=int, default=16)
    a = p.parse_args()
    assert run(a.fmt, a.prompts, a.steps) < 1e-5
