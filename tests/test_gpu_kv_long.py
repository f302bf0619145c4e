"""Attention over long runs of records on the GPU: every worker of the stream goes many times round its ring,
over the ends of pages, heads and sequences; sums of tens of thousands of terms.  The reference is 64-bit torch
on the same GPU."""
import math

import pytest
import torch

mmq = pytest.importorskip("block_quantized_int8_mmq_gb300")
pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
UNIT = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8, "f16": 2.0 ** -11}


def make_records(pages, heads, page, dim, gen, lowest):
    """Records of normal keys, values of codes lowest .. 127, and what they stand for: f64 [heads, tokens, dim]
    of page after page."""
    n = page // 32
    data = torch.zeros((pages, heads, n, 64 * dim + 16), dtype=torch.uint8, device="cuda")
    kc = torch.randn((pages, heads, n, 32 * dim), device="cuda", generator=gen).mul_(32).round_().clamp_(-127, 127)
    vc = torch.randint(lowest, 128, (pages, heads, n, 32 * dim), device="cuda", generator=gen)
    scales = torch.full((pages, heads, n, 2), 0.03, device="cuda")
    if lowest < 0:
        scales *= torch.rand(scales.shape, device="cuda", generator=gen) + 0.5
    data[..., :32 * dim] = kc.to(torch.int8).view(torch.uint8)
    data[..., 32 * dim:64 * dim] = vc.to(torch.int8).view(torch.uint8)
    data[..., 64 * dim:64 * dim + 8] = scales.view(torch.uint8)

    def values(codes, which):
        x = codes.double() * scales[..., which:which + 1].double()
        return x.view(pages, heads, n, 32, dim).transpose(0, 1)  # [heads, pages, n, 32, dim]

    return data, values(kc, 0), values(vc, 1)


def int32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("seqs,new", [(356, 1), (356, 4), (356, 6), (40, 130)])
def test_f32_sums_of_long_runs(dim, seqs, new):
    """f32 rows over 65500 tokens each (shared pages), values of one sign and of nearly one size: what is lost
    in adding them up shows.  Bound, of |out|:
      2^-19 (4 + S) spread  the weights' own errors (as in the other tests), which move the output by what the
                            values differ from it: spread = (127 - 96) / 96
      2^-22                 weights as two f16 terms
      2^-20                 a record's products (256 keys of the tiles) in the tensor cores, which round
                            towards zero
      2 * 6 sqrt(n / 3) 2^-23 / sqrt(12)   six deviations of n additions rounded to nearest, the sum of the
                            values and that of the weights, growing evenly; n: two a record of a unit at most"""
    gen = torch.Generator(device="cuda").manual_seed(dim + new)
    length, page, group = 65500, 256, 4
    pages = -(-length // page)
    data, k, v = make_records(pages, 1, page, dim, gen, 96)
    k, v = (x[0].reshape(-1, dim) for x in (k, v))
    table = torch.arange(pages, device="cuda", dtype=torch.int32)[None].repeat(seqs, 1)
    batch = mmq.KVBatch(int32([new * i for i in range(seqs + 1)]), int32([length] * seqs), table, seqs * new, new)
    q = torch.randn((seqs * new, group, dim), device="cuda", generator=gen) * 0.3
    out = mmq.mmq_kv_attend(mmq.KVCache(data), batch, q, scale=1 / math.sqrt(dim))
    torch.cuda.synchronize()
    assert mmq.mmq_get_device_error() == 0
    n = 2 * -(-length // 32)
    for b in range(0, seqs, max(1, seqs // 9)):
        for t in {0, new // 2, new - 1}:
            end, x = length - new + t + 1, q[b * new + t].double()
            s = x @ k[:end].T / math.sqrt(dim)
            want = s.softmax(-1) @ v[:end]
            big = float((x.abs() @ k[:end].abs().T).max()) / math.sqrt(dim)
            bound = 2.0 ** -19 * (4 + big) * (127 - 96) / 96 + 2.0 ** -22 + 2.0 ** -20 + \
                12 * math.sqrt(n / 3) * 2.0 ** -23 / math.sqrt(12) + UNIT["f32"]
            off = float(((out[b * new + t].double() - want) / want).abs().max())
            assert off <= bound, f"2^{math.log2(off):.1f} off, 2^{math.log2(bound):.1f} allowed"
